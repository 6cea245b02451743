"""Measured cases of the tokens' way to their experts and back, and of the FP8 expert products over ragged groups.

Operators (`kind` of a case):
  group      token-expert pairs in expert order: offsets, the row of each pair and the pair of each row (moe_group)
  dispatch   tokens copied to the rows of their experts, and the gradient back (moe_dispatch, moe_combine)
  combine    rows back to tokens with the routing weights applied, and its gradients (moe_combine, moe_combine_grad)
  product    ragged expert product on e4m3 operands with a scale for each block of 128 (grouped_gemm_fp8)
  linear     a training step's expert product in FP8: output, gradient of the rows and of the weights (grouped_linear_fp8)

The plain forms are elementary torch operations in fp32: ragged groups padded to the largest one and multiplied as a batch.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ZIPF = 1.1


# ------------------------------------------------------------------ cases
def _group(name, T, k, E, zipf):
    return {"name": name, "kind": "group", "T": T, "k": k, "E": E, "zipf": zipf}


def _dispatch(name, T, k, H, dtype):
    return {"name": name, "kind": "dispatch", "T": T, "k": k, "E": 64, "H": H, "dtype": dtype, "zipf": False}


def _combine(name, T, k, H, dtype, grad, dropped):
    return {"name": name, "kind": "combine", "T": T, "k": k, "E": 64, "H": H, "dtype": dtype, "grad": grad, "dropped": dropped,
            "zipf": False}


def _product(name, R, E, N, K, dtype, e8m0, zipf):
    return {"name": name, "kind": "product", "R": R, "E": E, "N": N, "K": K, "dtype": dtype, "e8m0": e8m0, "zipf": zipf}


def _linear(name, R, E, N, K, dtype, zipf):
    return {"name": name, "kind": "linear", "R": R, "E": E, "N": N, "K": K, "dtype": dtype, "zipf": zipf}


def listed():
    return [
        # one decode step of 64 tokens, top-8 of 256: latency
        _group("group_decode", 64, 8, 256, False),
        # a prefill of 8192 tokens, routing as uneven as Zipf's law
        _group("group_prefill", 8192, 8, 256, True),
        # the small test layer (16 tokens, top-4): latency
        _dispatch("dispatch_tiny", 16, 4, 256, "fp16"),
        # hidden states of 8192 tokens to their 8 experts, and the gradient back
        _dispatch("dispatch_prefill", 8192, 8, 7168, "bf16"),
        # a decode step's expert outputs back to 64 tokens
        _combine("combine_decode", 64, 8, 7168, "bf16", False, False),
        # the same in a training step of 8192 tokens, with gradients of rows and routing weights
        _combine("combine_train", 8192, 8, 7168, "bf16", True, False),
        # fp32 rows of an odd width, a third of the pairs with experts held elsewhere
        _combine("combine_odd", 1003, 6, 1160, "fp32", True, True),
        # one token's 8 experts of 256, gate and up, a checkpoint's fp32 scales: 248 experts without rows
        _product("product_token", 8, 256, 4096, 7168, "bf16", False, False),
        # the down projection of a 64-token decode step, top-8 of 256
        _product("product_decode", 512, 256, 7168, 2048, "bf16", False, False),
        # gate and up of a prefill of 8192 tokens a GPU, 32 local experts of 256
        _product("product_prefill", 65536, 32, 4096, 7168, "bf16", False, False),
        # a training step of the same layer at half the tokens: three products and their quantisations
        _linear("linear_train", 32768, 32, 4096, 7168, "bf16", False),
        # skewed routing with experts that get nothing, sizes off the tile and off the block
        _linear("linear_skew", 5003, 48, 1008, 1168, "fp16", True),
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["group", "dispatch", "combine", "product", "linear"])
    dtype = rng.choice(["bf16", "fp16"])
    zipf = rng.random() < 0.3
    if kind == "group":
        k = rng.randint(1, 8)
        return _drop(_group("", _log(rng, 1, 32768), k, max(k, _log(rng, 4, 512)), zipf))
    if kind in ("dispatch", "combine"):
        k, H = rng.randint(1, 8), _log(rng, 64, 7168, 8)
        T = _log(rng, 1, min(32768, 8192 * 8 * 7168 // (2 * k * H)))
        if kind == "dispatch":
            return _drop(_dispatch("", T, k, H, rng.choice([dtype, "fp32"])))
        return _drop(_combine("", T, k, H, rng.choice([dtype, "fp32"]), rng.random() < 0.7, rng.random() < 0.4))
    if kind == "product":
        E, K = _log(rng, 2, 256), _log(rng, 128, 7168, 16)
        N = _log(rng, 128, min(7168, 256 * 7168 * 2048 // (E * K)), 8)
        return _drop(_product("", _log(rng, 1, 32768 if not zipf else 8192), E, N, K, dtype, rng.random() < 0.5, zipf))
    E, N, K = _log(rng, 2, 64), _log(rng, 128, 4096, 16), _log(rng, 128, 4096, 16)
    return _drop(_linear("", _log(rng, 16, 16384 if not zipf else 8192), E, N, K, dtype, zipf))


def _drop(c):
    return {k: v for k, v in c.items() if k != "name"}


def _popularity(E, zipf):
    """Share of the pairs each expert is expected to get, most popular first."""
    p = torch.arange(1, E + 1, dtype=torch.float64) ** (-_ZIPF if zipf else 0.0)
    return p / p.sum()


def work(case):
    if case["kind"] == "group":
        n = case["T"] * case["k"]
        return {"bytes": 4 * n + 8 * n + 4 * (case["E"] + 1), "flops": n}
    if case["kind"] in ("dispatch", "combine"):
        T, H, b = case["T"], case["H"], 4 if case["dtype"] == "fp32" else 2
        n = T * case["k"]
        live = n * 2 / 3 if case.get("dropped") else n
        if case["kind"] == "dispatch":
            return {"bytes": 2 * b * H * (T + n) + 2 * 4 * n, "flops": n * H}
        if not case["grad"]:
            return {"bytes": b * H * (T + live) + 8 * n, "flops": 2 * live * H}
        return {"bytes": b * H * (2 * T + 3 * live) + 20 * n, "flops": 5 * live * H}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    active = float((1 - (1 - _popularity(E, case["zipf"])) ** R).sum())
    if case["kind"] == "product":
        sb = 1 if case["e8m0"] else 4
        KB = -(-K // 128)
        scales = sb * (active * -(-N // 128) * KB + R * KB)
        return {"bytes": active * N * K + R * K + 2 * R * N + scales + 4 * (E + 1), "flops": 2 * R * N * K}
    return {"bytes": 2 * (active * N * K + 2 * R * K + 2 * R * N + E * N * K) + 4 * (E + 1), "flops": 6 * R * N * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 23)

    def normal(*shape, std=1.0, to=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(to)

    def popularity(E):
        return _popularity(E, case["zipf"])[torch.randperm(E, generator=torch.Generator().manual_seed(int(seed) + 5))].to(dev)

    st = {"case": case}
    if case["kind"] in ("group", "dispatch", "combine"):
        T, k, E = case["T"], case["k"], case["E"]
        held = E * 3 // 2 if case.get("dropped") else E
        # the k largest of noisy scores: distinct experts, the popular ones more often
        score = torch.rand((T, held), generator=gen, device=dev).log().neg().log().neg() + popularity(held).log().float()
        ids = score.topk(k, 1).indices.to(torch.int32)
        st["ids"] = torch.where(ids < E, ids, -1) if held > E else ids
        if case["kind"] == "group":
            return st
        dt, H = _DT[case["dtype"]], case["H"]
        st["rop"] = _plain_group(st["ids"], E)["row_of_pair"]
        if case["kind"] == "dispatch":
            st["x"], st["drows"] = normal(T, H, to=dt), normal(T * k, H, std=0.01, to=dt)
            return st
        st["rows"] = normal(T * k, H, to=dt)
        w = torch.rand((T, k), generator=gen, device=dev) + 0.1
        st["weights"] = w / w.sum(1, keepdim=True) * 2.5
        if case["grad"]:
            st["dout"] = normal(T, H, std=0.01, to=dt)
            st["d"] = torch.zeros((T * k, H), dtype=dt, device=dev)  # rows of dropped pairs stay as they are
        return st
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    counts = torch.bincount(torch.multinomial(popularity(E), R, replacement=True, generator=gen), minlength=E)
    st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    st["most"] = int(counts.max())  # rows of the largest group
    if case["kind"] == "linear":
        dt = _DT[case["dtype"]]
        st["x"], st["dy"] = normal(R, K, to=dt).requires_grad_(), normal(R, N, std=0.01, to=dt)
        w = torch.empty((E, N, K), dtype=dt, device=dev)
        for e in range(E):
            w[e] = normal(N, K, std=0.02)
        st["w"] = w.requires_grad_()
        return st
    st["x8"], st["xs"] = _pack(normal(R, K, to=torch.bfloat16), 1, case["e8m0"])
    NB, KB = -(-N // 128), -(-K // 128)
    st["w8"] = torch.empty((E, N, K), dtype=torch.uint8, device=dev)
    st["ws"] = torch.empty((E, NB, KB), dtype=torch.uint8 if case["e8m0"] else torch.float32, device=dev)
    for e in range(E):
        st["w8"][e], st["ws"][e] = _pack(normal(N, K, std=0.02), 128, case["e8m0"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return _own(case, state) if own else _plain(case, state)


def _own(case, st):
    import fp8_block_scaled_grouped_amd as m
    if case["kind"] == "group":
        offsets, row_of_pair, pair_of_row = m.moe_group(st["ids"], case["E"])
        return {"offsets": offsets, "row_of_pair": row_of_pair, "pair_of_row": pair_of_row}
    if case["kind"] == "dispatch":
        return {"rows": m.moe_dispatch(st["x"], st["rop"]), "dx": m.moe_combine(st["drows"], st["rop"])}
    if case["kind"] == "combine":
        res = {"out": m.moe_combine(st["rows"], st["rop"], st["weights"])}
        if case["grad"]:
            res["drows"], res["dw"] = m.moe_combine_grad(st["dout"], st["rows"], st["rop"], st["weights"], st["d"])
        return res
    if case["kind"] == "product":
        return m.grouped_gemm_fp8(st["x8"], st["xs"], st["w8"], st["ws"], st["offsets"], out_dtype=_DT[case["dtype"]])
    y = m.grouped_linear_fp8(st["x"], st["w"], st["offsets"])
    dx, dw = torch.autograd.grad(y, (st["x"], st["w"]), st["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw}


def _plain_group(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key, order = torch.sort(torch.where((flat >= 0) & (flat < E), flat, E), stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device)).to(torch.int32)
    place = torch.arange(T * k, dtype=torch.int32, device=ids.device)
    live = key < E
    rop = torch.empty_like(place)
    rop[order] = torch.where(live, place, -1)
    return {"offsets": offsets, "row_of_pair": rop.view(T, k), "pair_of_row": torch.where(live, order, -1).to(torch.int32)}


def _gathered(rows, rop):
    """fp32 rows of each token's pairs [T, k, H], zeros for dropped ones."""
    return torch.where((rop >= 0)[..., None], rows.float()[rop.clamp(min=0).long()], 0.0)


def _scattered(pairs, rop, into):
    """[T, k, H] to the pairs' rows of a copy of `into`; what dropped pairs bring goes to a row behind the last."""
    n = into.shape[0]
    out = torch.cat([into, into.new_zeros(1, into.shape[1])])
    at = torch.where(rop >= 0, rop, n).long().reshape(-1)
    out[at] = pairs.reshape(-1, into.shape[1]).to(into.dtype)
    return out[:n]


def _plain(case, st):
    if case["kind"] == "group":
        return _plain_group(st["ids"], case["E"])
    if case["kind"] == "dispatch":
        x, rop = st["x"], st["rop"]
        rows = _scattered(x[:, None, :].expand(-1, case["k"], -1), rop, x.new_zeros(rop.numel(), x.shape[1]))
        return {"rows": rows, "dx": _gathered(st["drows"], rop).sum(1).to(x.dtype)}
    if case["kind"] == "combine":
        rop, w, dt = st["rop"], st["weights"], _DT[case["dtype"]]
        y = _gathered(st["rows"], rop)
        res = {"out": (y * w[..., None]).sum(1).to(dt)}
        if case["grad"]:
            d = st["dout"].float()[:, None, :]
            res["drows"] = _scattered(w[..., None] * d, rop, st["d"])
            res["dw"] = (y * d).sum(-1)
        return res
    off, most, R = st["offsets"].long(), st["most"], case["R"]
    dt = _DT[case["dtype"]]
    if case["kind"] == "product":
        x = _unpack(st["x8"], st["xs"], 1)
        w = _unpack(st["w8"], st["ws"], 128)
        return _ragged_rows(torch.bmm(_padded(x, off, most), w.transpose(1, 2)), off, R).to(dt)
    with torch.no_grad():
        x, dy = st["x"].detach(), st["dy"]
        w = torch.stack([_unpack(*_pack(e, 128, True), 128) for e in st["w"].detach()])
        xr, dyr = _unpack(*_pack(x, 1, True), 1), _unpack(*_pack(dy, 1, True), 1)
        y = _ragged_rows(torch.bmm(_padded(xr, off, most), w.transpose(1, 2)), off, R).to(dt)
        dx = _ragged_rows(torch.bmm(_padded(dyr, off, most), w), off, R).to(dt)
        # scales of 128 rows by one column, the rows counted from their group's first
        most = -(-most // 128) * 128
        xc, dyc = (_columns(_padded(t, off, most)) for t in (x, dy))
        return {"y": y, "dx": dx, "dw": torch.bmm(dyc.transpose(1, 2), xc).to(dt)}


def _columns(p):
    """[E, n * 128, C] rounded to e4m3 with a power-of-two scale for each 128 rows of a column."""
    g = p.view(p.shape[0], -1, 128, p.shape[2])
    s = _scale(g.abs().amax(2, keepdim=True), True)[0]
    return ((g / s).to(torch.float8_e4m3fn).float() * s).view_as(p)


def _scale(amax, e8m0):
    """fp32 scales of groups with these largest magnitudes, and their stored form."""
    if not e8m0:
        # a quotient of tensors: by a Python number, torch multiplies by the reciprocal
        s = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
        return s, s
    m, ex = torch.frexp(amax)  # amax = m * 2^ex, m in [0.5, 1)
    ex = torch.where(amax == 0, 0, (ex - 9 + (m > 0.875).int()).clamp(-127, 127))
    return _two_to(ex).float(), (ex + 127).to(torch.uint8)


def _two_to(ex):
    """2^ex as fp64, put together from its bits: torch's pow and ldexp are a rounding off on the GPU."""
    return ((ex.long() + 1023) << 52).view(torch.float64)


def _pack(t, rows, e8m0):
    """[n, K] -> (e4m3 codes, scales of blocks of `rows` x 128); also how a checkpoint ships the weights of prepare()."""
    n, K = t.shape
    pad = torch.nn.functional.pad(t.float(), (0, -K % 128, 0, -n % rows))
    g = pad.view(pad.shape[0] // rows, rows, pad.shape[1] // 128, 128)
    s, stored = _scale(g.abs().amax((1, 3), keepdim=True), e8m0)
    q = (g / s).to(torch.float8_e4m3fn).view(torch.uint8).view_as(pad)[:n, :K].contiguous()
    return q, stored.view(g.shape[0], g.shape[2])


def _unpack(q, scale, rows):
    """Codes [.., n, K] and scales of blocks of `rows` x 128 -> fp32 values."""
    s = _two_to(scale.long() - 127).float() if scale.dtype == torch.uint8 else scale
    n, K = q.shape[-2:]
    s = s.repeat_interleave(rows, -2)[..., :n, :] if rows > 1 else s
    return q.view(torch.float8_e4m3fn).float().mul_(s.repeat_interleave(128, -1)[..., :K])


def _padded(t, off, most):
    """fp32 [R, C] rows grouped by expert -> [E, most, C], zeros past each group's end."""
    at = off[:-1, None] + torch.arange(most, device=t.device)[None, :]
    live = at < off[1:, None]
    return torch.where(live[..., None], t.float()[at.clamp(max=t.shape[0] - 1)], 0.0)


def _ragged_rows(p, off, R):
    """[E, most, C] -> [R, C]."""
    r = torch.arange(R, device=p.device)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return p[e, r - off[e]]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "group":
        return None  # whole numbers: the plain form's have to be met exactly
    if case["kind"] in ("dispatch", "combine"):
        return _exact_rows(case, st)
    off, dev = st["offsets"].tolist(), st["offsets"].device
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    y = torch.zeros((R, N), dtype=torch.float64, device=dev)
    if case["kind"] == "product":
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                w = _e4m3(st["w8"][e]) * _each(st["ws"][e], 128, N, K)
                y[a:b] = (_e4m3(st["x8"][a:b]) * _each(st["xs"][a:b], 1, b - a, K)) @ w.t()
        return y
    dx = torch.zeros((R, K), dtype=torch.float64, device=dev)
    dw = torch.zeros((E, N, K), dtype=torch.float64, device=dev)
    x, dy = st["x"].detach(), st["dy"]
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            w = _nearest(st["w"][e].detach(), 128, 128)
            y[a:b] = _nearest(x[a:b], 1, 128) @ w.t()
            dx[a:b] = _nearest(dy[a:b], 1, 128) @ w
            dw[e] = _nearest(dy[a:b], 128, 1).t() @ _nearest(x[a:b], 128, 1)
    return {"y": y, "dx": dx, "dw": dw}


def _exact_rows(case, st):
    """Pair by pair of the tokens, j after j."""
    rop, T, k = st["rop"].long(), case["T"], case["k"]
    if case["kind"] == "dispatch":
        rows = torch.zeros((T * k, case["H"]), dtype=torch.float64, device=rop.device)
        dx = torch.zeros((T, case["H"]), dtype=torch.float64, device=rop.device)
        for j in range(k):
            rows[rop[:, j]] = st["x"].double()
            dx += st["drows"][rop[:, j]].double()
        return {"rows": rows, "dx": dx}
    out = torch.zeros((T, case["H"]), dtype=torch.float64, device=rop.device)
    w = st["weights"].double()
    drows, dw = st["d"].double() if case["grad"] else None, torch.zeros_like(w)
    for j in range(k):
        t = torch.nonzero(rop[:, j] >= 0)[:, 0]
        r = rop[t, j]
        y = st["rows"][r].double()
        out[t] += w[t, j, None] * y
        if case["grad"]:
            d = st["dout"][t].double()
            drows[r] = w[t, j, None] * d
            dw[t, j] = (y * d).sum(1)
    return {"out": out, "drows": drows, "dw": dw} if case["grad"] else {"out": out}


def _e4m3(q):
    """Value of an e4m3 code: m * 2^-9 below 8, else (8 + m) * 2^(e - 10), bit 7 the sign."""
    c = (q % 128).double()
    e, m = torch.floor(c / 8), c % 8
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two_to(e - 10))
    return torch.where(q >= 128, -v, v)


def _each(scale, rows, n, K):
    s = _two_to(scale.double() - 127) if scale.dtype == torch.uint8 else scale.double()
    return s[torch.arange(n, device=s.device) // rows][:, torch.arange(K, device=s.device) // 128]


def _nearest(t, rows, cols):
    """Nearest e4m3 multiples of each rows x cols block's scale, the smallest power of two that keeps the block in +-448."""
    out = t.double()
    n, K = out.shape
    p = torch.nn.functional.pad(out, (0, -K % cols, 0, -n % rows))
    g = p.view(p.shape[0] // rows, rows, p.shape[1] // cols, cols)
    top = g.abs().amax((1, 3), keepdim=True)
    f, ex = torch.frexp(torch.where(top == 0, 448.0, top) / 448)
    s = _two_to((ex - (f == 0.5).int()).clamp(-127, 127))
    y = g / s
    step = _two_to(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(y / step) * step * s).view_as(p)[:n, :K]
