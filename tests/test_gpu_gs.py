"""Group-scaled 4-bit weights on the GPU: packer, values, and the linear layer
against their 64-bit definitions."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import binary_weight_transformer_b200 as bwt
import gs_reference as ref

pytestmark = pytest.mark.gpu
DT = {bwt.F32: torch.float32, bwt.BF16: torch.bfloat16}


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def weights(seed, N, K):
    return (np.random.default_rng(seed).standard_normal((N, K)) * 0.02).astype(np.float32)


def tokens(seed, M, K):
    rng = np.random.default_rng(seed)
    ld = -(-K // 16) * 16
    q = rng.integers(-128, 128, (M, ld)).astype(np.int8)  # bytes past K are ignored: left random
    s = (0.01 + rng.random(M)).astype(np.float32)
    return q, s


def check_pack(w, group, sdt, wdt=bwt.F32, ldw=None):
    N, K = w.shape
    t = cuda(w).to(DT[wdt])
    w = t.float().cpu().numpy()
    if ldw is not None:
        wide = torch.full((N, ldw), 9.0, dtype=DT[wdt], device="cuda")
        wide[:, :K] = t
        t = wide[:, :K]
    st = status_word()
    packed, s = bwt.lowbit_gs_pack(t, group, sdt, status=st)
    codes, scales = ref.quantise(w, group, sdt == bwt.BF16)
    assert np.array_equal(s.float().cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(packed.cpu().numpy(), ref.pack(codes, packed.shape[1]))
    for odt in (bwt.F32, bwt.BF16):
        v = bwt.lowbit_gs_unpack(packed, s, K, group, odt, status=st)
        want = codes.astype(np.float32) * np.repeat(scales, group, axis=1)[:, :K]
        want = want if odt == bwt.F32 else ref.bf16_round(want)
        assert np.array_equal(v.float().cpu().numpy(), want)
    assert st.item() == 0


@pytest.mark.parametrize("group", bwt.GS_GROUPS)
@pytest.mark.parametrize("sdt", [bwt.F32, bwt.BF16])
@pytest.mark.parametrize("N,K,ldw", [(1, 1, None), (3, 31, None), (5, 33, 37), (7, 256, None), (4, 1000, 1004),
                                     (9, 1001, None), (17, 2560, 2568)])
def test_pack_and_values(group, sdt, N, K, ldw):
    for wdt in (bwt.F32, bwt.BF16):
        check_pack(weights(N * K, N, K), group, sdt, wdt, ldw)


@pytest.mark.parametrize("sdt", [bwt.F32, bwt.BF16])
@pytest.mark.parametrize("size", [1.0, 3e-5, 1e-20, 1e-37, 3e-39, 2e-44, 3e37])
def test_pack_halves(sdt, size):
    """Weights on, and one step beside, every half of their group's scale, at
    ordinary, tiny, subnormal and huge sizes."""
    rng = np.random.default_rng(7)
    w = np.zeros((64, 32), np.float32)
    for n in range(64):
        top = np.float32(size * (1 + rng.random()))
        s = np.float32(top / np.float32(7))
        s = ref.bf16_round(np.array([s]))[0] if sdt == bwt.BF16 else s
        half = ((np.arange(30) % 7 + 0.5) * np.float64(s) * np.where(np.arange(30) % 2, 1, -1)).astype(np.float32)
        step = np.arange(30) % 3
        half = np.where(step == 1, np.nextafter(half, np.float32(np.inf)), half)
        half = np.where(step == 2, np.nextafter(half, np.float32(-np.inf)), half)
        w[n, 0], w[n, 1:31] = top, np.clip(half, -top, top)
    check_pack(w, 32, sdt)


@pytest.mark.parametrize("sdt", [bwt.F32, bwt.BF16])
@pytest.mark.parametrize("exponent", [0, -50, 60])
def test_pack_every_bf16_weight_below_a_maximum(sdt, exponent):
    """Every 8-bit significand as the group's maximum, with every bf16 weight
    from a 32nd of it upwards, both signs: among them all that lie exactly on a
    half of the quotient or of the scale."""
    rows = []
    for b in range(128, 256):
        v = np.array([a * 2.0 ** p for p in range(-5, 1) for a in range(128, 256)])
        v = v[v <= b]
        v = np.concatenate([v, np.zeros(-len(v) % 31)]).reshape(-1, 31)
        v[:, ::2] *= -1
        rows.append(np.concatenate([np.full((len(v), 1), float(b)), v], 1))
        rows.append(-rows[-1])
    check_pack((np.concatenate(rows) * 2.0 ** exponent).astype(np.float32), 32, sdt, bwt.BF16)


@pytest.mark.parametrize("odt", [bwt.F32, bwt.BF16])
@pytest.mark.parametrize("N,K,skip", [(1200, 9001, 0), (1200, 9002, 1), (40000, 250, 3), (2000, 5000, 1), (300, 31, 1)])
def test_large_ragged_rows(odt, N, K, skip):
    """Rows and bases without the alignment of wide accesses, at sizes where a
    thread decodes several words; what lies beside the rows is left alone."""
    group = 64
    w = torch.randn(N, K, device="cuda").to(DT[odt])
    wide = torch.full((N, K + 5), 3.0, dtype=DT[odt], device="cuda")
    inside = wide.flatten()[skip:skip + (N - 1) * (K + 5) + K].as_strided((N, K), (K + 5, 1))
    inside.copy_(w)
    packed, s = bwt.lowbit_gs_pack(inside, group)
    p2, s2 = bwt.lowbit_gs_pack(torch.nn.functional.pad(w, (0, -K % 8)), group)
    assert torch.equal(s, s2[:, :s.shape[1]]) and torch.equal(packed, p2[:, :packed.shape[1]])
    inside.fill_(7.0)
    bwt.lowbit_gs_unpack(packed, s, K, group, odt, w=inside)
    bits = torch.stack([(packed >> sh) & 15 for sh in (0, 4)], -1).view(N, -1, 4, 2).transpose(2, 3).reshape(N, -1)[:, :K]
    codes = (bits ^ 8).float() - 8  # word by word: four low nibbles, then the high ones
    want = (codes * s.repeat_interleave(group, 1)[:, :K]).to(DT[odt])
    assert torch.equal(inside, want)
    inside.fill_(3.0)
    assert (wide == 3.0).all()


def test_pack_zero_groups_and_signed_zero():
    w = weights(3, 4, 512)
    w[0] = 0.0
    w[1, 64:128] = -0.0
    w[2, 500:] = 0.0
    for group in bwt.GS_GROUPS:
        check_pack(w, group, bwt.F32)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_pack_reports_nonfinite(bad):
    w = weights(4, 3, 300)
    w[1, 299] = bad
    st = status_word()
    packed, s = bwt.lowbit_gs_pack(cuda(w), 64, status=st)
    assert bwt.status_flags(st) == [bwt.ERR_NONFINITE]
    codes, scales = ref.quantise(weights(4, 3, 300), 64, False)
    assert np.array_equal(packed.cpu().numpy()[[0, 2]], ref.pack(codes, packed.shape[1])[[0, 2]])
    assert np.array_equal(s.cpu().numpy()[:, :4], scales[:, :4])


def test_unpack_reports_reserved_and_unowned_bits():
    packed, s = bwt.lowbit_gs_pack(cuda(weights(5, 2, 36)), 32)
    for byte, value in ((3, 0x08), (3, 0x80), (16, 0x10)):  # code 3, code 7, a code past K = 36
        p = packed.clone()
        p[1, byte] = value
        st = status_word()
        v = bwt.lowbit_gs_unpack(p, s, 36, 32, status=st)
        assert bwt.status_flags(st) == [bwt.ERR_RESERVED_CODE]
        assert torch.isfinite(v).all()


def check_linear(M, K, N, group, sdt, odt, seed=0, stable=False, lds=None, ldy=None, ldp=None):
    rng = np.random.default_rng(seed + M + 3 * K + 7 * N)
    codes = rng.integers(-7, 8, (N, K)).astype(np.int8)
    G = bwt.gs_groups(K, group)
    scales = (0.001 + 0.01 * rng.random((N, G))).astype(np.float32)
    if sdt == bwt.BF16:
        scales = ref.bf16_round(scales)
    ldp = bwt.packed_ld(bwt.INT4, K) if ldp is None else ldp
    packed = ref.pack(codes, ldp)
    row = bwt.packed_row_bytes(bwt.INT4, K)
    packed[:, row:] = 0x5A  # bytes behind a row's codes carry no meaning
    q, s_x = tokens(seed + 1, M, K)
    s_g = cuda(scales).to(DT[sdt])
    if lds is not None:
        wide = torch.full((N, lds), 7.0, dtype=s_g.dtype, device="cuda")
        wide[:, :G] = s_g
        s_g = wide[:, :G]
    ldy = N if ldy is None else ldy
    y = torch.full((M, ldy), 77.0, dtype=DT[odt], device="cuda")
    st = status_word()
    args = (cuda(q), cuda(s_x), cuda(packed), s_g, group, odt)
    got = bwt.lowbit_gs_linear(*args, K=K, y=y[:, :N], status=st, weights_stable=stable)
    want, mag = ref.linear(q[:, :K], s_x, codes, scales, group)
    err = np.abs(got.double().cpu().numpy() - want)
    assert st.item() == 0
    assert (err <= ref.linear_bound(want, mag, G, odt == bwt.BF16)).all().item(), err.max()
    assert (y[:, N:] == 77.0).all()
    again = bwt.lowbit_gs_linear(*args, K=K)
    assert torch.equal(got, again)


@pytest.mark.parametrize("group", bwt.GS_GROUPS)
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("K,N", [(200, 33), (1280, 72)])
def test_linear_few_tokens(group, M, K, N):
    check_linear(M, K, N, group, bwt.F32 if M % 2 else bwt.BF16, bwt.F32)
    check_linear(M, K, N, group, bwt.BF16 if M % 2 else bwt.F32, bwt.BF16)


@pytest.mark.parametrize("group", bwt.GS_GROUPS)
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 16, 8), (2, 31, 9), (5, 127, 16), (3, 129, 5), (1, 9728, 24),
                                   (4, 2561, 40), (16, 4097, 31)])
def test_linear_edges(group, M, K, N):
    check_linear(M, K, N, group, bwt.F32, bwt.F32)


@pytest.mark.parametrize("M,K,N", [(40, 640, 96), (64, 1000, 300), (100, 2560, 200), (129, 333, 129), (300, 1280, 257),
                                   (512, 64, 1000), (700, 2080, 136)])
@pytest.mark.parametrize("group", bwt.GS_GROUPS)
def test_linear_many_tokens(M, K, N, group):
    check_linear(M, K, N, group, bwt.F32, bwt.F32)
    check_linear(M, K, N, group, bwt.BF16, bwt.BF16)


@pytest.mark.parametrize("M,K,N", [(100, 5000, 200), (129, 4096, 96), (300, 2560, 257), (40, 9728, 513), (200, 16385, 31)])
@pytest.mark.parametrize("group", bwt.GS_GROUPS)
def test_linear_deep(M, K, N, group):
    """Few tiles over a long K: each tile's K is split over several SM pairs."""
    check_linear(M, K, N, group, bwt.F32, bwt.F32)
    check_linear(M, K, N, group, bwt.BF16, bwt.BF16, ldy=N + 7)


@pytest.mark.parametrize("M", [1, 3, 40])
@pytest.mark.parametrize("K,group", [(98304, 64), (98560, 32), (bwt.GS_MAX_K, 256)])
def test_linear_longest_rows(M, K, group):
    """K at and past what the single-token kernel keeps in shared memory, and
    the largest.  Weights of -7 to 7 with 7s in every group pack to themselves."""
    N = 9
    gen = torch.Generator("cuda").manual_seed(K)
    w = torch.randint(-7, 8, (N, K), device="cuda", generator=gen).float()
    w[:, ::group] = 7
    q = torch.randint(-128, 128, (M, K), device="cuda", generator=gen, dtype=torch.int8)
    s_x = torch.rand(M, device="cuda", generator=gen) + 0.1
    packed, s_g = bwt.lowbit_gs_pack(w, group)
    assert (s_g == 1).all()
    s_g *= torch.rand(s_g.shape, device="cuda", generator=gen) + 0.1
    y = bwt.lowbit_gs_linear(q, s_x, packed, s_g, group)
    acc = (q.double().view(M, 1, -1, group) * w.double().view(1, N, -1, group)).sum(-1) * s_g.double()
    want, mag = acc.sum(-1) * s_x.double()[:, None], acc.abs().sum(-1) * s_x.double()[:, None]
    bound = ref.linear_bound(want.cpu().numpy(), mag.cpu().numpy(), K // group, False)
    assert (np.abs((y.double() - want).cpu().numpy()) <= bound).all()


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_linear_rows_past_32_bits(M):
    """Output rows so far apart that their offsets pass 2^31 elements."""
    N, K = 40, 1280
    ldy = 2 ** 31 // (M - 1) + 64 if M > 1 else N
    packed, s_g = bwt.lowbit_gs_pack(cuda(weights(5, N, K)), 64)
    q, s_x = (cuda(a) for a in tokens(6, M, K))
    want = bwt.lowbit_gs_linear(q, s_x, packed, s_g, 64)
    flat = torch.empty((M - 1) * ldy + N, device="cuda")
    y = flat.as_strided((M, N), (ldy, 1))
    bwt.lowbit_gs_linear(q, s_x, packed, s_g, 64, y=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_linear_operands_past_32_bits(M):
    """Rows of codes, packed weights and scales whose byte offsets pass 2^31."""
    N, K, group = 40, 1280, 64
    packed, s_g = bwt.lowbit_gs_pack(cuda(weights(5, N, K)), group)
    q, s_x = (cuda(a) for a in tokens(6, M, K))
    want = bwt.lowbit_gs_linear(q, s_x, packed, s_g, group)

    def apart(t, ld):
        flat = torch.empty((len(t) - 1) * ld + t.shape[1], dtype=t.dtype, device="cuda")
        far = flat.as_strided(t.shape, (ld, 1))
        far.copy_(t)
        return far

    far = [apart(packed, 2 ** 26), apart(s_g, 2 ** 25 + 1)]
    q = apart(q, (2 ** 31 // (M - 1) + 16) // 16 * 16) if M > 1 else q
    assert torch.equal(bwt.lowbit_gs_linear(q, s_x, *far, group, K=K), want)


def test_first_calls_inside_a_capture():
    """In a fresh process: what a kernel sets up on its first call may happen
    while a graph is captured."""
    code = """
import torch, binary_weight_transformer_b200 as bwt
torch.cuda.init()
w = torch.randn(600, 1280, device="cuda")
x = torch.randn(500, 1280, device="cuda")
e = torch.randint(0, 4, (500, 2), device="cuda", dtype=torch.int32)
r = torch.rand(500, 2, device="cuda")
bwt.lib()

def run():
    p, s = bwt.lowbit_gs_pack(w, 64)
    v = bwt.lowbit_gs_unpack(p, s, 1280, 64)
    q, sx = bwt.lowbit_act_quant(x)
    ys = [bwt.lowbit_gs_linear(q[:m], sx[:m], p, s, 64) for m in (1, 9, 500)]
    off, pos = bwt.lowbit_moe_plan(e, 4)
    qs, ss = bwt.lowbit_moe_gather(q, pos, s_x=sx)
    z = bwt.lowbit_gs_linear_experts(qs, ss, off, p.view(4, 150, -1), s.view(4, 150, -1), 64)
    y = bwt.lowbit_moe_combine(z, pos, r)
    return [v, *ys, y, *bwt.lowbit_moe_combine_backward(y, z, pos, r)]

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, want))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]


def test_unpack_words_past_32_bits():
    """More than 2^31 packed words (of 40 GB of values)."""
    N, K = 600_000, 32768
    if torch.cuda.mem_get_info()[0] < 70e9:
        pytest.skip("needs 70 GB")
    packed = torch.full((N, K // 2), 0x17, device="cuda", dtype=torch.uint8)  # codes 7 and 1
    packed[-1], packed[N // 2] = 0x2E, 0xF3
    s = torch.ones(N, K // 256, device="cuda", dtype=torch.bfloat16)
    v = bwt.lowbit_gs_unpack(packed, s, K, 256, bwt.BF16)
    low = [7.0] * 4 + [1.0] * 4
    for r, word in ((0, low), (N - 2, low), (N - 1, [-2.0] * 4 + [2.0] * 4), (N // 2, [3.0] * 4 + [-1.0] * 4)):
        assert torch.equal(v[r], torch.tensor(word * (K // 8), device="cuda", dtype=torch.bfloat16))
    del v
    torch.cuda.empty_cache()


def test_unpack_values_past_32_bits():
    N, K = 70000, 32768  # 2.3e9 values
    packed = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    packed[(packed & 15) == 8] = 0x11
    packed[(packed >> 4) == 8] = 0x11
    s = torch.rand(N, K // 256, device="cuda") + 0.5
    v = bwt.lowbit_gs_unpack(packed, s, K, 256, bwt.BF16)
    for r in (0, N // 2, N - 1):
        one = bwt.lowbit_gs_unpack(packed[r:r + 1], s[r:r + 1], K, 256, bwt.BF16)
        assert torch.equal(v[r:r + 1], one)
    again, s2 = bwt.lowbit_gs_pack(v, 256)
    r = slice(N - 2, N)
    p1, s1 = bwt.lowbit_gs_pack(v[r].contiguous(), 256)
    assert torch.equal(again[r], p1) and torch.equal(s2[r], s1)


@pytest.mark.parametrize("M", [1, 12, 200])
def test_linear_strides(M):
    check_linear(M, 500, 50, 64, bwt.BF16, bwt.BF16, stable=True, lds=11, ldy=57, ldp=320)
    check_linear(M, 512, 64, 128, bwt.F32, bwt.F32, lds=5, ldy=65, ldp=256)


@pytest.mark.parametrize("M", [3, 16, 200])
def test_linear_extreme_codes_and_scales(M):
    """All codes at their limits (the largest integer sums), and scales of
    very different sizes side by side, zeros among them."""
    K, N, group = 2048, 40, 256
    q = np.full((M, K), -128, np.int8)
    codes = np.full((N, K), 7, np.int8)
    codes[::2] = -7
    rng = np.random.default_rng(2)
    scales = (10.0 ** rng.integers(-30, 4, (N, K // group))).astype(np.float32)
    scales[3] = 0.0
    s_x = np.full(M, 0.5, np.float32)
    packed = cuda(ref.pack(codes, K // 2))
    got = bwt.lowbit_gs_linear(cuda(q), cuda(s_x), packed, cuda(scales), group)
    want, mag = ref.linear(q, s_x, codes, scales, group)
    assert (np.abs(got.double().cpu().numpy() - want) <= ref.linear_bound(want, mag, K // group, False)).all()
    assert (got[:, 3] == 0).all()


@pytest.mark.parametrize("M,K", [(1, 336), (16, 336), (400, 336), (200, 4240)])
def test_linear_infinite_scale_follows_the_sum(M, K):
    """An infinite scale of a group whose integer sum is not zero gives an
    infinity, in the row's first group (whatever pads K) and in its last."""
    N, group = 40, 32
    q, s_x = np.ones((M, K), np.int8), np.ones(M, np.float32)
    packed = cuda(ref.pack(np.full((N, K), 3, np.int8), bwt.packed_ld(bwt.INT4, K)))
    for at in (0, K // group):
        s = torch.ones(N, bwt.gs_groups(K, group), device="cuda")
        s[5, at] = float("inf")
        y = bwt.lowbit_gs_linear(cuda(q), cuda(s_x), packed, s, group)
        assert torch.isposinf(y[:, 5]).all()
        y[:, 5] = 3 * K
        assert (y == 3 * K).all()


def test_linear_infinite_scale_stays_in_its_rows():
    w, (q, s_x) = weights(8, 24, 256), tokens(9, 5, 256)
    packed, s = bwt.lowbit_gs_pack(cuda(w), 64)
    clean = bwt.lowbit_gs_linear(cuda(q), cuda(s_x), packed, s, 64)
    s2, x2 = s.clone(), cuda(s_x)
    s2[7, 1] = float("inf")
    x2[3] = float("nan")
    got = bwt.lowbit_gs_linear(cuda(q), x2, packed, s2, 64)
    rows, cols = [0, 1, 2, 4], [n for n in range(24) if n != 7]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[:, 7]).any()


def test_linear_equals_int4_layer_with_one_scale():
    """With every group scale of a row equal, the layer is lowbit_linear's
    4-bit one: integer sums of the row times one scale."""
    N, K, M = 96, 1024, 6
    packed, s_w = bwt.lowbit_pack(cuda(weights(1, N, K)), bwt.INT4)
    q, s_x = tokens(2, M, K)
    want = bwt.lowbit_linear(cuda(q), cuda(s_x), packed, s_w, bwt.INT4, N, bwt.F32, K=K).double()
    s_g = s_w[:, None].expand(N, K // 128).contiguous()
    got = bwt.lowbit_gs_linear(cuda(q), cuda(s_x), packed, s_g, 128).double()
    codes = bwt.lowbit_unpack(packed, K, bwt.INT4).cpu().numpy()
    _, mag = ref.linear(q, s_x, codes, s_g.cpu().numpy(), 128)
    # lowbit_linear rounds three times (conversion, scale product, product)
    assert ((got - want).abs().cpu().numpy() <= ref.linear_bound(want.cpu().numpy(), mag, 8, False) + 3 * ref.U32 * mag).all()


@pytest.mark.parametrize("M", [1, 16, 160])
def test_layer_in_a_graph_and_on_another_stream(M):
    """Prologue, product and the pack before it, captured once and replayed on
    new inputs; and two calls at once on two streams."""
    N, K = 264, 640
    x = torch.randn(M, K, device="cuda")
    w = torch.randn(N, K, device="cuda")

    def layer(x, w):
        packed, s = bwt.lowbit_gs_pack(w, 64, bwt.BF16)
        q, s_x = bwt.lowbit_act_quant_ex(x, norm=bwt.NORM_RMS)
        return bwt.lowbit_gs_linear(q, s_x, packed, s, 64, bwt.BF16)

    eager = layer(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, w)
    graph.replay()
    assert torch.equal(out, eager)
    x.copy_(torch.randn(M, K, device="cuda"))
    w.copy_(torch.randn(N, K, device="cuda"))
    graph.replay()
    assert torch.equal(out, layer(x, w))

    packed, s = bwt.lowbit_gs_pack(w, 64)
    q, s_x = bwt.lowbit_act_quant(x)
    want = bwt.lowbit_gs_linear(q, s_x, packed, s, 64)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i].append(bwt.lowbit_gs_linear(q, s_x, packed, s, 64, stream=st, y=torch.empty_like(want)))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for half in got for g in half)


@pytest.mark.parametrize("M,K,waits", [(300, 2560, True), (60, 9728, False), (200, 320, False), (128, 9728, True)])
def test_timeout_is_reported_and_the_context_survives(M, K, waits):
    """Every pipeline wait of the tcgen05 kernel is bounded: with the bound
    lowered to one cycle the first wait that does not succeed at once gives up,
    the status says so, and the kernel ends by itself; afterwards, with the
    bound restored, the same call is right again.  (The two small
    products run on the warp-level kernel, which has no such waits: estimated
    9.4 + 0.33 * 6.8 * 4 = 18 against 4.2 + 2.6 + 0.7 + 19 * 0.67 = 20 us, and
    4.7 + 0.33 * 0.22 * 13 = 5.6 against 4.2 + 0.7 + 3 * 0.67 = 6.9.)"""
    N = 700
    packed, s_g = bwt.lowbit_gs_pack(cuda(weights(5, N, K)), 64)
    q, s_x = (cuda(a) for a in tokens(6, M, K))
    want = bwt.lowbit_gs_linear(q, s_x, packed, s_g, 64)
    torch.cuda.synchronize()
    bwt.set_wait_limit(1)
    try:
        st = status_word()
        y = bwt.lowbit_gs_linear(q, s_x, packed, s_g, 64, status=st)
        torch.cuda.synchronize()
        assert bwt.status_flags(st) == ([bwt.ERR_TIMEOUT] if waits else [])
        assert waits or torch.equal(y, want)
    finally:
        bwt.set_wait_limit(0)
    st = status_word()
    assert torch.equal(bwt.lowbit_gs_linear(q, s_x, packed, s_g, 64, status=st), want)
    assert st.item() == 0


@pytest.mark.parametrize("M", [16, 100, 700])
def test_two_products_at_once(M):
    """Products of all kernels interleaved on three streams, each with operands
    of its own."""
    N, K, group = 520, 2560, 128
    calls = []
    for i in range(3):
        packed, s_g = bwt.lowbit_gs_pack(cuda(weights(i, N, K)), group)
        q, s_x = (cuda(a) for a in tokens(10 + i, M, K))
        calls.append((q, s_x, packed, s_g, group))
    want = [bwt.lowbit_gs_linear(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[torch.empty_like(want[0]) for _ in range(6)] for _ in calls]
    for j in range(6):
        for st, c, g in zip(streams, calls, got):
            bwt.lowbit_gs_linear(*c, stream=st, y=g[j])
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)


def test_wrappers_refuse_on_the_gpu():
    """Shapes, strides and types of CUDA tensors that the C side cannot see."""
    q, s_x = (cuda(a) for a in tokens(1, 4, 64))
    packed, s = bwt.lowbit_gs_pack(cuda(weights(1, 8, 64)), 32)
    for args, kw, err in (((q, s_x[:3], packed, s, 32), {}, ValueError), ((q, s_x, packed, s, 64), {}, ValueError),
                          ((q, s_x, packed, s, 48), {}, ValueError), ((q, s_x, packed, s, 32), dict(K=65), ValueError),
                          ((q, s_x, packed, s, 32), dict(K=0), ValueError),
                          ((q, s_x, packed[:, :16], s, 32), {}, ValueError),
                          ((q, s_x, packed, s.half(), 32), {}, TypeError), ((q, s_x.double(), packed, s, 32), {}, TypeError),
                          ((q, s_x, packed, s, 32, bwt.I32), {}, ValueError),
                          ((q, s_x, packed, s, 32), dict(y=torch.empty(4, 9, device="cuda")), ValueError),
                          ((q, s_x, packed, s, 32), dict(y=torch.empty(8, 4, device="cuda").T), ValueError),
                          ((q, s_x, packed, s, 32), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")), ValueError),
                          ((q[:, ::2], s_x, packed, s, 32), dict(K=16), ValueError),
                          ((q, s_x, packed.cpu(), s, 32), {}, ValueError)):
        with pytest.raises(err):
            bwt.lowbit_gs_linear(*args, **kw)
    with pytest.raises(bwt.LowbitError):  # rows of codes that overlap
        bwt.lowbit_gs_linear(q[:1].expand(4, 64), s_x, packed, s, 32)
    with pytest.raises(ValueError):  # packed rows of a wider buffer
        bwt.lowbit_gs_pack(cuda(weights(1, 8, 64)), 32, packed=torch.empty(8, 64, dtype=torch.uint8, device="cuda")[:, :32])
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        bwt.lowbit_moe_gather(q, pos[:3])
    with pytest.raises(ValueError):
        bwt.lowbit_moe_gather(q, pos, s_out=s_x)
    with pytest.raises(TypeError):
        bwt.lowbit_moe_combine(q, pos)
    with pytest.raises(ValueError):
        bwt.lowbit_moe_combine(s, pos, torch.ones(4, 4, device="cuda")[:, ::2])
