"""Expert routing and the experts' products on the GPU, against their 64-bit
definitions; and the whole path as an expert layer runs it."""
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


def route(seed, T, k, E, drop=0.0, skew=False):
    rng = np.random.default_rng(seed)
    e = (E * rng.random((T, k)) ** (4 if skew else 1)).astype(np.int64)
    return np.where(rng.random((T, k)) < drop, -1, e)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 3), (5, 2, 8), (33, 3, 40), (300, 4, 64), (2048, 1, 7),
                                   (2049, 1, 1024), (5000, 3, 16), (20000, 2, 128), (9000, 8, 1), (8192, 8, 64),
                                   (16384, 4, 1024), (30000, 3, 5)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_plan(T, k, E, drop, wide):
    e = route(T + E, T, k, E, drop, skew=T % 2 == 0)
    st = status_word()
    off, pos = bwt.lowbit_moe_plan(cuda(e.astype(np.int64 if wide else np.int32)), E, status=st)
    want_off, want_pos = ref.plan(e, E)
    assert st.item() == 0
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(pos.cpu().numpy(), want_pos)


@pytest.mark.parametrize("T", [3, 4000])
def test_plan_all_dropped_and_bad_ids(T):
    off, pos = bwt.lowbit_moe_plan(torch.full((T, 2), -1, dtype=torch.int32, device="cuda"), 9)
    assert (off == 0).all() and (pos == -1).all()
    e = route(1, T, 2, 9)
    e[T // 2, 1], e[0, 0] = 9, 2 ** 40
    st = status_word()
    off, pos = bwt.lowbit_moe_plan(cuda(e), 9, status=st)
    assert bwt.status_flags(st) == [bwt.ERR_INVALID_ARG]
    want_off, want_pos = ref.plan(e, 9)
    assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(pos.cpu().numpy(), want_pos)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16, torch.float32, torch.float64])
@pytest.mark.parametrize("width,ld", [(1, 1), (3, 5), (64, 64), (100, 102), (1280, 1280), (1001, 1001), (5000, 5008),
                                      (1004, 1004), (1002, 1002), (4098, 4098)])
def test_gather(dtype, width, ld):
    T, k, E = 37, 3, 5
    off, pos = (cuda(a) for a in ref.plan(route(width, T, k, E, 0.3), E))
    x = (100 * torch.randn(T, ld, device="cuda")).to(dtype)[:, :width]
    s = torch.rand(T, device="cuda")
    out = torch.full((T * k, ld), 55, device="cuda").to(dtype)
    s_out = torch.full((T * k,), -1.0, device="cuda")
    st = status_word()
    bwt.lowbit_moe_gather(x, pos, s_x=s, out=out[:, :width], s_out=s_out, status=st)
    n = int(off[-1])
    p = pos.flatten().long()
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    assert st.item() == 0
    assert torch.equal(out[p[p >= 0], :width], x[token[p >= 0]])
    assert torch.equal(s_out[p[p >= 0]], s[token[p >= 0]])
    assert (out[n:] == 55).all() and (out[:, width:] == 55).all() and (s_out[n:] == -1).all()


def test_gather_skips_rows_past_the_end():
    pos = torch.tensor([[0, 7], [1, 4]], dtype=torch.int32, device="cuda")
    x, out, st = torch.ones(2, 16, device="cuda"), torch.zeros(4, 16, device="cuda"), status_word()
    guard = torch.zeros(4, 16, device="cuda")
    bwt.lowbit_moe_gather(x, pos, out=out, status=st)
    assert bwt.status_flags(st) == [bwt.ERR_INVALID_ARG]
    assert (out[:2] == 1).all() and (out[2:] == 0).all() and (guard == 0).all()
    for fn in (lambda s: bwt.lowbit_moe_combine(out, pos, status=s),
               lambda s: bwt.lowbit_moe_combine_backward(x, out, pos, torch.ones(2, 2, device="cuda"),
                                                         d_ys=torch.zeros(4, 16, device="cuda"), status=s)):
        st.zero_()
        fn(st)
        assert bwt.status_flags(st) == [bwt.ERR_INVALID_ARG]


def combine_ref(ys, pos, w):
    v = ys[np.maximum(pos, 0)] * (pos >= 0)[..., None]
    return (v * w[..., None]).sum(1), (np.abs(v) * np.abs(w)[..., None]).sum(1)


@pytest.mark.parametrize("dt", [bwt.F32, bwt.BF16])
@pytest.mark.parametrize("T,k,K,ld", [(1, 1, 1, 1), (3, 2, 7, 9), (40, 5, 64, 64), (16, 2, 1280, 1280),
                                      (9, 8, 2560, 2560), (300, 4, 1001, 1003), (700, 9, 520, 520), (2, 3, 9000, 9000),
                                      (60, 5, 1002, 1002), (90, 3, 1004, 1004), (7, 2, 4098, 4098),
                                      (2500, 2, 1001, 1001)])
def test_combine_and_gradients(dt, T, k, K, ld):
    E = 6
    rng = np.random.default_rng(T + K)
    _, pos = ref.plan(route(T * K, T, k, E, 0.25), E)
    pos[0] = -1 if T > 2 else pos[0]  # a token whose slots are all dropped
    used = pos[pos >= 0]
    rows = T * k + 3
    ys = cuda(rng.standard_normal((rows, ld)).astype(np.float32)).to(DT[dt])[:, :K]
    dy = cuda(rng.standard_normal((T, ld)).astype(np.float32)).to(DT[dt])[:, :K]
    w = rng.standard_normal((T, k)).astype(np.float32)
    tp, tw = cuda(pos), cuda(w)
    u = ref.UBF if dt == bwt.BF16 else 0.0
    for weight in (w, None):
        y = torch.full((T, ld), 3.0, dtype=DT[dt], device="cuda")
        bwt.lowbit_moe_combine(ys, tp, tw if weight is not None else None, y=y[:, :K])
        want, mag = combine_ref(ys.double().cpu().numpy(), pos, np.ones_like(w, dtype=np.float64) if weight is None else w.astype(np.float64))
        # k multiply-adds, each rounding at most mag; the result's own rounding
        e = k * ref.U32 * mag * (1 + 1e-3)
        assert (np.abs(y[:, :K].double().cpu().numpy() - want) <= e + u * (np.abs(want) + e)).all()
        assert (y[:, K:] == 3.0).all()

    d_ys = torch.full((rows, ld), 5.0, dtype=DT[dt], device="cuda")
    _, d_w = bwt.lowbit_moe_combine_backward(dy, ys, tp, tw, d_ys=d_ys[:, :K])
    t_of = np.repeat(np.arange(T), k)[pos.reshape(-1) >= 0]
    want = (cuda(w.reshape(-1)[pos.reshape(-1) >= 0])[:, None] * dy.float()[cuda(t_of)]).to(DT[dt])
    assert torch.equal(d_ys[cuda(used).long(), :K], want)  # one product, one rounding: the same bits
    rest = np.setdiff1d(np.arange(rows), used)
    assert (d_ys[cuda(rest)] == 5.0).all() and (d_ys[:, K:] == 5.0).all()
    v = ys.double().cpu().numpy()[np.maximum(pos, 0)] * (pos >= 0)[..., None]
    prod = v * dy.double().cpu().numpy()[:, None, :]
    # a sum of K products in any order: at most K roundings of the sum of |products|
    assert (np.abs(d_w.double().cpu().numpy() - prod.sum(-1)) <= (K + 2) * ref.U32 * np.abs(prod).sum(-1)).all()
    assert (d_w.cpu().numpy()[pos < 0] == 0).all()


def test_gradients_against_differences():
    """L = <dy, combine(ys, w)> is linear in ys and in w: a difference of L is
    exact but for rounding.  gather's gradient the same way."""
    T, k, K, E, h = 24, 3, 96, 5, 0.5
    g = torch.Generator("cuda").manual_seed(3)
    _, pos = ref.plan(route(5, T, k, E, 0.2), E)
    tp = cuda(pos)
    ys = torch.randn(T * k, K, device="cuda", generator=g)
    w = torch.randn(T, k, device="cuda", generator=g)
    dy = torch.randn(T, K, device="cuda", generator=g)
    d_ys, d_w = bwt.lowbit_moe_combine_backward(dy, ys, tp, w, d_ys=torch.zeros_like(ys))
    loss = lambda ys, w: (dy.double() * bwt.lowbit_moe_combine(ys, tp, w).double()).sum()  # noqa: E731
    size = (dy.abs().double() * bwt.lowbit_moe_combine(ys.abs(), tp, w.abs()).double()).sum().item()
    tol = 4 * (k + 2) * ref.U32 * size / h  # two losses, each off by (k + 2) roundings of their terms
    for t, j in ((0, 0), (7, 2), (23, 1)):
        w2 = w.clone()
        w2[t, j] += h
        assert abs((loss(ys, w2) - loss(ys, w)).item() / h - d_w[t, j].item()) <= tol
    for r, c in ((0, 0), (11, 95), (30, 40)):
        y2 = ys.clone()
        y2[r, c] += h
        assert abs((loss(y2, w) - loss(ys, w)).item() / h - d_ys[r, c].item()) <= tol
    x = torch.randn(T, K, device="cuda", generator=g)
    d_out = torch.randn(T * k, K, device="cuda", generator=g)
    d_x = bwt.lowbit_moe_combine(d_out, tp)
    gather = lambda x: (d_out.double() * bwt.lowbit_moe_gather(x, tp, out=torch.zeros_like(d_out)).double()).sum()  # noqa: E731
    for t, c in ((0, 0), (9, 50), (23, 95)):
        x2 = x.clone()
        x2[t, c] += h
        assert abs((gather(x2) - gather(x)).item() / h - d_x[t, c].item()) <= tol


def expert_weights(seed, E, N, K, group, sdt):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-7, 8, (E, N, K)).astype(np.int8)
    scales = (0.001 + 0.01 * rng.random((E, N, bwt.gs_groups(K, group)))).astype(np.float32)
    if sdt == bwt.BF16:
        scales = ref.bf16_round(scales)
    packed = np.stack([ref.pack(c, bwt.packed_ld(bwt.INT4, K)) for c in codes])
    return codes, scales, cuda(packed), cuda(scales).to(DT[sdt])


def check_experts(counts, K, N, group, sdt, odt, spare=3, seed=0, strided=False):
    E, n = len(counts), int(sum(counts))
    codes, scales, packed, s_g = expert_weights(seed, E, N, K, group, sdt)
    if strided:  # experts further apart than their weights, rows of scales too
        wide = torch.full((E, N + 2, packed.shape[2] + 32), 0x5A, dtype=torch.uint8, device="cuda")
        wide[:, :N, :packed.shape[2]] = packed
        packed = wide[:, :N, :packed.shape[2]]
        ws = torch.full((E, N + 1, s_g.shape[2] + 3), 9.0, dtype=s_g.dtype, device="cuda")
        ws[:, :N, :s_g.shape[2]] = s_g
        s_g = ws[:, :N, :s_g.shape[2]]
    rng = np.random.default_rng(seed + 1)
    rows = n + spare
    q = rng.integers(-128, 128, (rows, -(-K // 16) * 16)).astype(np.int8)
    s_x = (0.1 + rng.random(rows)).astype(np.float32)
    s_x[n:] = np.nan
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.full((rows, N + 5), 66.0, dtype=DT[odt], device="cuda")
    st = status_word()
    got = bwt.lowbit_gs_linear_experts(cuda(q), cuda(s_x), cuda(off), packed, s_g, group, odt, K=K, y=y[:, :N], status=st)
    assert st.item() == 0
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        want, mag = ref.linear(q[a:b, :K], s_x[a:b], codes[e], scales[e], group)
        err = np.abs(got[a:b].double().cpu().numpy() - want)
        assert (err <= ref.linear_bound(want, mag, scales.shape[2], odt == bwt.BF16)).all().item(), (e, err.max())
    assert (y[n:] == 66.0).all() and (y[:, N:] == 66.0).all()


@pytest.mark.parametrize("group", bwt.GS_GROUPS)
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 9, 1], [2] * 16, [0, 0, 0, 0, 40], [17, 8, 33, 1, 0, 5]])
def test_experts_few_rows(counts, group):
    check_experts(counts, 330, 40, group, bwt.F32, bwt.F32)
    check_experts(counts, 1280, 24, group, bwt.BF16, bwt.BF16)


@pytest.mark.parametrize("group", bwt.GS_GROUPS)
@pytest.mark.parametrize("counts", [[200, 0, 131, 400], [1, 900, 3], [64, 65, 63, 128, 1, 0, 0, 127], [300]])
def test_experts_many_rows(counts, group):
    check_experts(counts, 328, 136, group, bwt.BF16, bwt.BF16)
    check_experts(counts, 1024, 257, group, bwt.F32, bwt.F32, spare=0)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("E", [33, 300, bwt.MOE_MAX_EXPERTS])
def test_many_experts(E, rows):
    """As many experts as there may be, every third without rows."""
    rng = np.random.default_rng(E)
    check_experts([0 if e % 3 == 0 else int(rng.integers(rows, 2 * rows + 1)) for e in range(E)], 64, 24, 32, bwt.F32, bwt.F32)


@pytest.mark.parametrize("rows", [3, 90])
def test_one_expert_takes_all_rows(rows):
    """The kernel is chosen for evenly spread rows; it is right for others."""
    check_experts([0] * 20 + [20 * rows] + [0] * 11, 640, 72, 64, bwt.BF16, bwt.BF16)


@pytest.mark.parametrize("counts", [[3, 0, 5], [150, 0, 260]])
def test_experts_strides(counts):
    check_experts(counts, 500, 72, 64, bwt.BF16, bwt.F32, strided=True)
    check_experts(counts, 500, 72, 128, bwt.F32, bwt.BF16, strided=True, spare=200)


@pytest.mark.parametrize("counts", [[3, 0, 5], [150, 40, 200]])
def test_experts_apart_past_32_bits(counts):
    """Experts whose weights and scales lie more than 2^31 bytes apart."""
    K, N, group = 640, 40, 64
    _, _, packed, s_g = expert_weights(4, 3, N, K, group, bwt.F32)
    q = torch.randint(-128, 128, (sum(counts), K), dtype=torch.int8, device="cuda")
    s_x = torch.rand(sum(counts), device="cuda")
    off = cuda(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    want = bwt.lowbit_gs_linear_experts(q, s_x, off, packed, s_g, group)

    def apart(t, step):
        far = torch.empty(2 * step + t[0].numel(), dtype=t.dtype, device="cuda").as_strided(t.shape, (step, *t.stride()[1:]))
        far.copy_(t)
        return far

    got = bwt.lowbit_gs_linear_experts(q, s_x, off, apart(packed, 2 ** 31 + 64), apart(s_g, 2 ** 30 + 3), group)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dt", [bwt.F32, bwt.BF16])
def test_routing_rows_past_32_bits(dt):
    """Rows of gather, combine and its gradient more than 2^31 elements in."""
    T, k, K, E = 6, 2, 1001, 3
    _, pos = ref.plan(route(8, T, k, E), E)
    tp, w = cuda(pos), torch.rand(T, k, device="cuda")
    x, dy = (torch.randn(T, K, device="cuda").to(DT[dt]) for _ in range(2))

    def apart(rows):
        ld = 2 ** 31 // (rows - 1) + 5
        return torch.zeros((rows - 1) * ld + K, dtype=DT[dt], device="cuda").as_strided((rows, K), (ld, 1))

    ys = bwt.lowbit_moe_gather(x, tp)
    far_ys = apart(T * k)
    bwt.lowbit_moe_gather(x, tp, out=far_ys)
    assert torch.equal(far_ys, ys)
    y, far_y = bwt.lowbit_moe_combine(ys, tp, w), apart(T)
    bwt.lowbit_moe_combine(far_ys, tp, w, y=far_y)
    assert torch.equal(far_y, y)
    d_ys, d_w = bwt.lowbit_moe_combine_backward(dy, ys, tp, w)
    far_y.copy_(dy)
    far_d, far_w = bwt.lowbit_moe_combine_backward(far_y, far_ys, tp, w, d_ys=apart(T * k))
    assert torch.equal(far_d, d_ys)
    size = (ys.float().abs().max() * dy.float().abs().max()).item() * K
    assert (far_w - d_w).abs().max().item() <= 2 * (K + 2) * ref.U32 * size  # two orders of one sum


@pytest.mark.parametrize("rows", [16, 400])
def test_experts_without_tokens(rows):
    y = torch.full((rows, 32), 4.0, device="cuda")
    _, _, packed, s_g = expert_weights(0, 5, 32, 64, 32, bwt.F32)
    bwt.lowbit_gs_linear_experts(torch.zeros(rows, 64, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda"),
                                 torch.zeros(6, dtype=torch.int32, device="cuda"), packed, s_g, 32, y=y)
    assert (y == 4.0).all()


@pytest.mark.parametrize("scale", [1, 60])
@pytest.mark.parametrize("offsets", [[0, 3, 9], [0, 5, 2], [-4, 2, 6], [6, 6, 2 ** 31 - 1]])
def test_experts_bad_offsets_stay_in_bounds(offsets, scale):
    rows = 6 * scale
    off = np.array([min(o * scale, 2 ** 31 - 1) for o in offsets], np.int32)
    _, _, packed, s_g = expert_weights(0, 2, 16, 64, 32, bwt.F32)
    buf = torch.full((rows + 8, 16), 8.0, device="cuda")
    st = status_word()
    bwt.lowbit_gs_linear_experts(torch.ones(rows, 64, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda"),
                                 cuda(off), packed, s_g, 32, y=buf[4:rows + 4], status=st)
    assert bwt.status_flags(st) == [bwt.ERR_INVALID_ARG]
    assert (buf[:4] == 8.0).all() and (buf[rows + 4:] == 8.0).all()


def expert_layer(x, experts, weights, packed, s_g, group, odt=bwt.F32):
    """Codes once per token, sorted, every expert's product, and back."""
    E = packed.shape[0]
    q, s_x = bwt.lowbit_act_quant(x)
    offsets, pos = bwt.lowbit_moe_plan(experts, E)
    qs, s_xs = bwt.lowbit_moe_gather(q, pos, s_x=s_x)
    ys = bwt.lowbit_gs_linear_experts(qs, s_xs, offsets, packed, s_g, group, odt, K=x.shape[1])
    return bwt.lowbit_moe_combine(ys, pos, weights), ys, pos


@pytest.mark.parametrize("T,k,E", [(1, 2, 4), (12, 2, 8), (700, 3, 6)])
def test_expert_layer(T, k, E):
    """The run of all of them against the definition in 64 bits, then captured
    into a graph and replayed on other tokens and another routing."""
    K, N, group = 384, 200, 64
    codes, scales, packed, s_g = expert_weights(1, E, N, K, group, bwt.F32)
    value = codes.astype(np.float64) * np.repeat(scales.astype(np.float64), group, axis=2)[..., :K]
    x = torch.randn(T, K, device="cuda")
    e = cuda(route(2, T, k, E, 0.1).astype(np.int32))
    w = torch.rand(T, k, device="cuda")

    def check(y, x, e, w):
        q, s = bwt.lowbit_act_quant(x)
        xd = q[:, :K].double().cpu().numpy() * s.double().cpu().numpy()[:, None]
        want, mag = np.zeros((T, N)), np.zeros((T, N))
        for t, row in enumerate(e.cpu().numpy()):
            for j, ex in enumerate(row):
                if ex >= 0:
                    wt = float(w[t, j])
                    want[t] += wt * (value[ex] @ xd[t])
                    mag[t] += abs(wt) * (np.abs(value[ex]) @ np.abs(xd[t]))
        bound = ref.linear_bound(want, mag, scales.shape[2], False) + (k + 1) * ref.U32 * mag
        assert (np.abs(y.double().cpu().numpy() - want) <= bound).all()

    y, _, _ = expert_layer(x, e, w, packed, s_g, group)
    check(y, x, e, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_layer(x, e, w, packed, s_g, group)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, _ = expert_layer(x, e, w, packed, s_g, group)
    for seed in (4, 5):
        x.copy_(torch.randn(T, K, device="cuda"))
        e.copy_(cuda(route(seed, T, k, E, 0.3, skew=True).astype(np.int32)))
        w.copy_(torch.rand(T, k, device="cuda"))
        graph.replay()
        check(out, x, e, w)


def test_backward_of_the_way_there_and_back():
    """Gradients through combine and gather around a linear map of the sorted
    rows, against autograd on the same plain operations in fp64; captured and
    replayed beside the eager result."""
    T, k, E, K = 50, 2, 7, 128
    _, pos = ref.plan(route(9, T, k, E, 0.2), E)
    tp, keep = cuda(pos), cuda(pos >= 0)
    x, w, dy = torch.randn(T, K, device="cuda"), torch.rand(T, k, device="cuda"), torch.randn(T, K, device="cuda")
    scale = torch.rand(T * k, 1, device="cuda")

    def backward():
        xs = bwt.lowbit_moe_gather(x, tp, out=torch.zeros(T * k, K, device="cuda"))
        d_ys, d_w = bwt.lowbit_moe_combine_backward(dy, xs * scale, tp, w, d_ys=torch.zeros_like(xs))
        return bwt.lowbit_moe_combine(d_ys * scale, tp), d_w

    d_x, d_w = backward()
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    xs = xd[:, None, :].expand(T, k, K) * scale.double()[tp.clamp(min=0).long()]
    ((xs * (wd * keep)[..., None]).sum(1) * dy.double()).sum().backward()
    # products of three factors and a sum of k terms; a dot of K terms
    assert ((d_x - xd.grad).abs() <= (k + 3) * ref.U32 * (dy.abs() * k).double()).all()
    size = (xs.detach().abs() * dy.abs().double()[:, None]).sum(-1)
    assert ((d_w - wd.grad).abs() <= (K + 4) * ref.U32 * size).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, gw = backward()
    graph.replay()
    assert torch.equal(gx, d_x) and torch.equal(gw, d_w)
