"""Measured cases of the group-scaled 4-bit operators and of the expert routing around them.

Five operators, each with a plain form in elementary torch operations (``own``
false) and as calls of the package (``own`` true):

* ``pack``     weights -> 4-bit codes with one scale per group of a row, and back to values
* ``linear``   y = s_x * sum over groups of s_g * (q . c), from int8 token codes
* ``sort``     token rows copied into expert order (a stable sort), and the gradient
* ``experts``  the group-scaled product of every expert with its own rows
* ``combine``  expert rows back in token order with routing weights applied, and the gradients

A packed row holds eight 4-bit two's-complement codes per 32-bit word: code k
is in byte k % 4 of word k // 8, in the low nibble for k % 8 < 4 and the high
one otherwise.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16, "i8": torch.int8}
SIZES = {F32: 4, BF16: 2, "i8": 1}
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a 4B-class feed-forward weight converted once from an fp32 checkpoint
        dict(name="pack 9728x2560", op="pack", N=9728, K=2560, group=128, w=F32, s=F32, out=F32),
        # a small layer with a ragged last group, bf16 checkpoint, short groups
        dict(name="pack 300x1001", op="pack", N=300, K=1001, group=32, w=BF16, s=BF16, out=BF16),
        # one decode step of one sequence
        dict(name="linear M=1", op="linear", M=1, K=2560, N=9728, group=128, s=F32, out=BF16),
        # the smallest call: a few tokens, odd sizes, latency counts
        dict(name="linear M=3 odd", op="linear", M=3, K=200, N=333, group=64, s=BF16, out=F32),
        # decode of a batch of 16 sequences through the long rows of a down projection
        dict(name="linear M=16", op="linear", M=16, K=9728, N=2560, group=128, s=BF16, out=BF16),
        # prefill of 8192 tokens
        dict(name="linear M=8192", op="linear", M=8192, K=2560, N=9728, group=128, s=F32, out=BF16),
        # routing of a small decode batch, int8 codes with their scales
        dict(name="sort T=16", op="sort", T=16, k=2, E=8, K=1280, x="i8", grad=False, drop=0.0),
        # a training batch: bf16 rows sorted and the gradient brought back, some slots dropped
        dict(name="sort T=8192 grad", op="sort", T=8192, k=4, E=64, K=2560, x=BF16, grad=True, drop=0.05),
        # experts of a decode batch: few rows each, bound by the weights
        dict(name="experts T=16", op="experts", T=16, k=2, E=8, K=1280, N=3584, group=128, s=F32, out=BF16, drop=0.0),
        # experts of a prefill: hundreds of rows each, uneven
        dict(name="experts T=4096", op="experts", T=4096, k=2, E=16, K=1280, N=3584, group=64, s=BF16, out=BF16,
             drop=0.02),
        # the way back for a decode batch
        dict(name="combine T=16", op="combine", T=16, k=2, K=1280, E=8, x=BF16, grad=False, drop=0.0),
        # the way back for a training batch with the gradients of rows and weights
        dict(name="combine T=8192 grad", op="combine", T=8192, k=4, K=2560, E=64, x=BF16, grad=True, drop=0.05),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["pack", "linear", "linear", "sort", "experts", "experts", "combine"])
    group = rng.choice([32, 64, 128, 256])
    s, out = rng.choice([F32, BF16]), rng.choice([F32, BF16])
    if op == "pack":
        K = _log(rng, 32, 9728)
        N = min(_log(rng, 16, 9728), 9728 * 2560 // K)
        return dict(op=op, N=N, K=K, group=group, w=rng.choice([F32, BF16]), s=s, out=out)
    if op == "linear":
        K, N = _log(rng, 64, 9728), _log(rng, 16, 9728)
        M = max(1, min(_log(rng, 1, 8192), 8192 * 2560 * 9728 // (K * N)))
        return dict(op=op, M=M, K=K, N=N, group=group, s=s, out=out)
    E = _log(rng, 2, 128)
    k = rng.randint(1, min(E, 8))
    drop = rng.choice([0.0, 0.0, 0.05, 0.5])
    K = _log(rng, 64, 4096)
    if op == "experts":
        N = max(16, min(_log(rng, 16, 3584), 16 * 3584 * 1280 // (E * K)))
        T = max(1, min(_log(rng, 1, 8192), 4 * 8192 * 1280 * 3584 // (k * K * N)))
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, group=group, s=s, out=out, drop=drop)
    x = rng.choice([F32, BF16, "i8"]) if op == "sort" else rng.choice([F32, BF16])
    T = max(1, min(_log(rng, 1, 8192), 8192 * 4 * 2560 * 2 // (k * K * SIZES[x])))
    return dict(op=op, T=T, k=k, E=E, K=K, x=x, grad=x != "i8" and rng.random() < 0.5, drop=drop)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _words(codes):
    """Packed rows of int codes [..., K] (K a multiple of 32): uint8 [..., K / 2]."""
    v = (codes & 15).reshape(*codes.shape[:-1], -1, 2, 4).to(torch.uint8)
    return (v[..., 0, :] | (v[..., 1, :] << 4)).flatten(-2).contiguous()


def _quantise(w, group, s_dtype):
    """Codes and group scales of w[..., K]: scale absmax / 7 in 32 bits, rounded to its type; code rint(w / scale).

    Both quotients are taken in 64 bits: a scale that is one step off moves the codes next to a half."""
    K = w.shape[-1]
    pad = -K % group
    v = torch.nn.functional.pad(w.float(), (0, pad)).unflatten(-1, (-1, group))
    s = (v.abs().amax(-1).double() / 7.0).float().to(s_dtype)
    d = s.double().unsqueeze(-1)
    c = torch.where(d > 0, (v.double() / torch.where(d > 0, d, 1.0)).round().clamp(-7, 7), 0.0)
    return c.to(torch.int8).flatten(-2)[..., :K], s


def _codes(g, rows, K):
    """int8 codes and scales of normal activations with 0.5% outliers, row stride a multiple of 16."""
    x = torch.randn(rows, K, generator=g, device=DEVICE)
    x = torch.where(torch.rand(rows, K, generator=g, device=DEVICE) < 0.005, x * 10, x)
    top = x.abs().amax(1)
    q = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.int8, device=DEVICE)
    q[:, :K] = (x * 127 / top[:, None]).round().clamp(-128, 127).to(torch.int8)
    return q, top / 127


def _weights(g, shape, K, group, s_dtype):
    w = 0.02 * torch.randn(*shape, K, generator=g, device=DEVICE)
    c, s = _quantise(w, group, s_dtype)
    return _words(torch.nn.functional.pad(c, (0, -K % 32))), s


def _route(g, T, k, E, drop):
    """Distinct experts per token, some more popular than others; a share `drop` of the slots carries -1."""
    score = torch.randn(T, E, generator=g, device=DEVICE) + 0.7 * torch.randn(E, generator=g, device=DEVICE)
    top, e = score.topk(k, dim=1)
    e = torch.where(torch.rand(T, k, generator=g, device=DEVICE) < drop, -1, e)
    return e.to(torch.int32), top.softmax(1).float()


def _plan(e, E):
    """(offsets, pos) of a stable sort of the slots by expert, dropped slots left out."""
    flat = e.flatten().long()
    counts = (flat[:, None] == torch.arange(E, device=e.device)).sum(0)
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    order = torch.where(flat < 0, E, flat).sort(stable=True).indices
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(flat.numel(), device=e.device)
    return off.to(torch.int32), torch.where(flat < 0, -1, pos).to(torch.int32).reshape(e.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    c, op = dict(case), case["op"]
    if op == "pack":
        c["weight"] = (0.02 * torch.randn(c["N"], c["K"], generator=g, device=DEVICE)).to(DTYPES[c["w"]])
        c["values"] = torch.empty(c["N"], c["K"], dtype=DTYPES[c["out"]], device=DEVICE)
        return c
    if op == "linear":
        c["q"], c["s_x"] = _codes(g, c["M"], c["K"])
        c["packed"], c["s_g"] = _weights(g, (c["N"],), c["K"], c["group"], DTYPES[c["s"]])
        c["y"] = torch.empty(c["M"], c["N"], dtype=DTYPES[c["out"]], device=DEVICE)
        return c
    T, k, E, K = c["T"], c["k"], c["E"], c["K"]
    c["e"], c["weights"] = _route(g, T, k, E, c["drop"])
    if op == "sort":
        if c["x"] == "i8":
            c["rows"], c["s_x"] = _codes(g, T, K)
            c["s_out"] = torch.zeros(T * k, device=DEVICE)
        else:
            c["rows"], c["s_x"], c["s_out"] = torch.randn(T, K, generator=g, device=DEVICE).to(DTYPES[c["x"]]), None, None
        # rows behind the last expert's are not written: zero here, in every form
        c["sorted"] = torch.zeros(T * k, c["rows"].shape[1], dtype=c["rows"].dtype, device=DEVICE)
        c["d_sorted"] = torch.randn(T * k, K, generator=g, device=DEVICE).to(c["rows"].dtype) if c["grad"] else None
        return c
    c["offsets"], c["pos"] = _plan(c["e"], E)
    if op == "experts":
        c["q"], c["s_x"] = _codes(g, T * k, K)
        c["packed"], c["s_g"] = _weights(g, (E, c["N"]), K, c["group"], DTYPES[c["s"]])
        c["y"] = torch.zeros(T * k, c["N"], dtype=DTYPES[c["out"]], device=DEVICE)
    else:
        c["ys"] = torch.randn(T * k, K, generator=g, device=DEVICE).to(DTYPES[c["x"]])
        c["y"] = torch.empty(T, K, dtype=DTYPES[c["x"]], device=DEVICE)
        c["dy"] = torch.randn(T, K, generator=g, device=DEVICE).to(DTYPES[c["x"]]) if c["grad"] else None
        c["d_ys"] = torch.zeros(T * k, K, dtype=DTYPES[c["x"]], device=DEVICE) if c["grad"] else None
    return c


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(c):
    return (_own if own else _plain)[c["op"]](c)


def _unpacked(packed, K):
    """Codes [..., K] of packed rows, as fp32."""
    b = packed.unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -2).flatten(-3)[..., :K].float()
    return n - 16 * (n >= 8)


def _values(packed, s_g, K, group):
    s = s_g.float().repeat_interleave(group, -1)[..., :K]
    return _unpacked(packed, K) * s


def _plain_pack(c):
    codes, s = _quantise(c["weight"], c["group"], DTYPES[c["s"]])
    values = codes.float() * s.float().repeat_interleave(c["group"], -1)[:, :c["K"]]
    return {"values": values.to(DTYPES[c["out"]]), "scales": s}


def _plain_linear(c):
    K = c["K"]
    y = c["q"][:, :K].float() @ _values(c["packed"], c["s_g"], K, c["group"]).T
    return (y * c["s_x"][:, None]).to(DTYPES[c["out"]])


def _gathered(rows, pos):
    """rows [R, K] at pos [T, k] in 32 bits; zero where pos is negative."""
    v = rows.float()[pos.clamp(min=0).long()]
    return v * (pos >= 0).unsqueeze(-1)


def _plain_sort(c):
    off, pos = _plan(c["e"], c["E"])
    t = torch.arange(c["T"], device=pos.device)[:, None].expand_as(pos)[pos >= 0]
    p = pos[pos >= 0].long()
    got = {"offsets": off, "pos": pos, "rows": torch.zeros_like(c["sorted"]).index_copy_(0, p, c["rows"][t])}
    if c["s_x"] is not None:
        got["rows"] = got["rows"][:, :c["K"]]
        got["scales"] = torch.zeros_like(c["s_out"]).index_copy_(0, p, c["s_x"][t])
    if c["grad"]:
        got["d_rows"] = _gathered(c["d_sorted"], pos).sum(1).to(c["rows"].dtype)
    return got


def _plain_experts(c):
    K, E = c["K"], c["E"]
    off = c["offsets"].long()
    rows = torch.arange(c["q"].shape[0], device=off.device)
    e = torch.bucketize(rows, off[1:], right=True)
    rows, e = rows[e < E], e[e < E]
    # every expert's rows padded to the longest, one batched product
    at = rows - off[e]
    x = torch.zeros(E, int((off[1:] - off[:-1]).max()), K, device=off.device)
    x[e, at] = c["q"][rows, :K].float()
    y = torch.bmm(x, _values(c["packed"], c["s_g"], K, c["group"]).transpose(1, 2))
    full = torch.zeros_like(c["y"])
    full[rows] = (y[e, at] * c["s_x"][rows, None]).to(full.dtype)
    return full


def _plain_combine(c):
    v = _gathered(c["ys"], c["pos"])
    got = {"y": (v * c["weights"].unsqueeze(-1)).sum(1).to(c["ys"].dtype)}
    if c["grad"]:
        dy = c["dy"].float().unsqueeze(1)
        d = (c["weights"].unsqueeze(-1) * dy).to(c["ys"].dtype)
        keep = c["pos"] >= 0
        got["d_ys"] = torch.zeros_like(c["d_ys"]).index_copy_(0, c["pos"][keep].long(), d[keep])
        got["d_weights"] = (v * dy).sum(-1)
    return got


_plain = {"pack": _plain_pack, "linear": _plain_linear, "sort": _plain_sort, "experts": _plain_experts,
          "combine": _plain_combine}


def _kind(name):
    import binary_weight_transformer_b200 as bwt
    return bwt.F32 if name == F32 else bwt.BF16


def _own_pack(c):
    import binary_weight_transformer_b200 as bwt
    packed, s = bwt.lowbit_gs_pack(c["weight"], c["group"], _kind(c["s"]))
    return {"values": bwt.lowbit_gs_unpack(packed, s, c["K"], c["group"], _kind(c["out"]), w=c["values"]), "scales": s}


def _own_linear(c):
    import binary_weight_transformer_b200 as bwt
    return bwt.lowbit_gs_linear(c["q"], c["s_x"], c["packed"], c["s_g"], c["group"], _kind(c["out"]), K=c["K"],
                                y=c["y"])


def _own_sort(c):
    import binary_weight_transformer_b200 as bwt
    off, pos = bwt.lowbit_moe_plan(c["e"], c["E"])
    bwt.lowbit_moe_gather(c["rows"], pos, s_x=c["s_x"], out=c["sorted"], s_out=c["s_out"])
    got = {"offsets": off, "pos": pos, "rows": c["sorted"]}
    if c["s_x"] is not None:
        got["rows"] = got["rows"][:, :c["K"]]
        got["scales"] = c["s_out"]
    if c["grad"]:
        got["d_rows"] = bwt.lowbit_moe_combine(c["d_sorted"], pos)
    return got


def _own_experts(c):
    import binary_weight_transformer_b200 as bwt
    return bwt.lowbit_gs_linear_experts(c["q"], c["s_x"], c["offsets"], c["packed"], c["s_g"], c["group"],
                                        _kind(c["out"]), K=c["K"], y=c["y"])


def _own_combine(c):
    import binary_weight_transformer_b200 as bwt
    got = {"y": bwt.lowbit_moe_combine(c["ys"], c["pos"], c["weights"], y=c["y"])}
    if c["grad"]:
        got["d_ys"], got["d_weights"] = bwt.lowbit_moe_combine_backward(c["dy"], c["ys"], c["pos"], c["weights"],
                                                                        d_ys=c["d_ys"])
    return got


_own = {"pack": _own_pack, "linear": _own_linear, "sort": _own_sort, "experts": _own_experts, "combine": _own_combine}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op == "pack":
        n, groups = c["N"] * c["K"], c["N"] * -(-c["K"] // c["group"])
        return {"bytes": n * SIZES[c["w"]] + n // 2 + groups * SIZES[c["s"]] + n * SIZES[c["out"]], "flops": 3 * n}
    if op in ("linear", "experts"):
        rows = c["M"] if op == "linear" else max(1, round(c["T"] * c["k"] * (1 - c["drop"])))
        sets = 1 if op == "linear" else min(c["E"], rows)
        weight = c["N"] * (c["K"] // 2 + -(-c["K"] // c["group"]) * SIZES[c["s"]])
        return {"bytes": rows * (c["K"] + 4) + sets * weight + rows * c["N"] * SIZES[c["out"]],
                "flops": 2 * rows * c["K"] * c["N"]}
    T, slots, row = c["T"], c["T"] * c["k"], c["K"] * SIZES[c["x"]]
    kept = max(1, round(slots * (1 - c["drop"])))
    if op == "sort":
        n = 8 * slots + (T + kept) * (row + (4 if c["x"] == "i8" else 0)) + (kept + T) * row * c["grad"]
        return {"bytes": n, "flops": slots + kept * c["K"] * c["grad"]}
    n = 8 * slots + kept * row + T * row + c["grad"] * (T * row + kept * row + 4 * slots)
    return {"bytes": n, "flops": kept * c["K"] * (2 + 3 * c["grad"])}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _wide(packed, s_g, K, group):
    """float64 weights of packed rows: each code sign-extended out of its 32-bit word, times its group's scale."""
    word = packed.contiguous().view(torch.int32).long()
    k = torch.arange(K, device=packed.device)
    shift = (k % 4) * 8 + (k % 8) // 4 * 4
    nibble = (word[..., k // 8] >> shift) & 15
    return torch.where(nibble > 7, nibble - 16, nibble).double() * s_g.double()[..., k // group]


def exact(case, seed):
    c, op = prepare(case, seed), case["op"]
    if op == "pack":
        w, group = c["weight"].double(), c["group"]
        at = torch.arange(c["K"], device=w.device) // group
        top = torch.zeros(c["N"], int(at[-1]) + 1, dtype=torch.float64, device=w.device)
        top.scatter_reduce_(1, at.expand_as(w), w.abs(), "amax")
        s = (top / 7).float().to(DTYPES[c["s"]]).double()  # as it is held
        d = s[:, at]
        v = torch.where(d > 0, torch.round(w / d).clamp(-7, 7) * d, torch.zeros_like(w))
        return {"values": v, "scales": s}
    if op == "linear":
        return c["q"][:, :c["K"]].double() @ _wide(c["packed"], c["s_g"], c["K"], c["group"]).mT * c["s_x"].double()[:, None]
    if op == "experts":
        y = torch.zeros(c["y"].shape, dtype=torch.float64, device=c["y"].device)
        off = c["offsets"].tolist()
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            x = c["q"][a:b, :c["K"]].double() * c["s_x"][a:b, None].double()
            y[a:b] = x @ _wide(c["packed"][e], c["s_g"][e], c["K"], c["group"]).mT
        return y
    if op == "sort":
        e = c["e"].flatten().tolist()
        order = [i for x in range(c["E"]) for i in range(len(e)) if e[i] == x] if len(e) * c["E"] <= 1 << 22 else \
            [i for i in sorted(range(len(e)), key=lambda i: e[i]) if e[i] >= 0]
        token = torch.tensor([i // c["k"] for i in order], dtype=torch.long, device=c["e"].device)
        got = {"offsets": None, "pos": None, "rows": None}
        if c["x"] != "i8":
            got["rows"] = torch.zeros(c["sorted"].shape, dtype=torch.float64, device=token.device)
            got["rows"][:len(order)] = c["rows"].double()[token]
        else:
            got["scales"] = torch.zeros(c["s_out"].shape, dtype=torch.float64, device=token.device)
            got["scales"][:len(order)] = c["s_x"].double()[token]
        if c["grad"]:
            d = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=token.device)
            got["d_rows"] = d.index_add_(0, token, c["d_sorted"][:len(order)].double())
        return got
    y = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=c["ys"].device)
    got = {"y": y}
    if c["grad"]:
        got["d_ys"] = torch.zeros(c["ys"].shape, dtype=torch.float64, device=y.device)
        got["d_weights"] = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=y.device)
    for j in range(c["k"]):
        t = torch.nonzero(c["pos"][:, j] >= 0).flatten()
        p, w = c["pos"][t, j].long(), c["weights"][t, j].double()[:, None]
        y[t] += w * c["ys"][p].double()
        if c["grad"]:
            got["d_ys"][p] = w * c["dy"][t].double()
            got["d_weights"][t, j] = torch.einsum("tk,tk->t", c["dy"][t].double(), c["ys"][p].double())
    return got
