"""Measured cases of the 4-bit weight operators and the ragged expert products.

Operators (`kind` of a case):
  fp4        pack a weight matrix to 4 bits with group scales and unpack it again (fp4_quant_groups, fp4_dequant_groups)
  gemm       linear layer on 4-bit weights, few rows (gemm_fp4_groupscale)
  experts    the same for rows grouped by expert (grouped_gemm_fp4)
  fwd, bwd   ragged expert products on 16-bit operands and their two gradients (grouped_gemm, grouped_gemm_dgrad,
             grouped_gemm_wgrad)

The plain forms are elementary torch operations in fp32: 4-bit codes through a table of their 16 values, ragged groups padded to
the largest one and multiplied as a batch.
"""
import math

import torch

own = False

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ZIPF = 1.1


# ------------------------------------------------------------------ cases
def _fp4(name, rows, K, dtype, group, e8m0):
    return {"name": name, "kind": "fp4", "rows": rows, "K": K, "dtype": dtype, "group": group, "e8m0": e8m0}


def _gemm(name, M, N, K, dtype, group, e8m0):
    return {"name": name, "kind": "gemm", "M": M, "N": N, "K": K, "dtype": dtype, "group": group, "e8m0": e8m0}


def _experts(name, R, E, N, K, dtype, group, e8m0, zipf):
    return {"name": name, "kind": "experts", "R": R, "E": E, "N": N, "K": K, "dtype": dtype, "group": group, "e8m0": e8m0,
            "zipf": zipf}


def _ragged(name, kind, R, E, N, K, dtype, dw, zipf):
    return {"name": name, "kind": kind, "R": R, "E": E, "N": N, "K": K, "dtype": dtype, "dw": dw, "zipf": zipf}


def listed():
    return [
        # one projection's weights packed at load time
        _fp4("pack_linear", 2048, 7168, "bf16", 128, False),
        # the gate/up weights of 32 local experts, OCP MX scales
        _fp4("pack_experts", 32 * 4096, 7168, "bf16", 32, True),
        # decode of one sequence through a small projection: latency
        _gemm("linear_1", 1, 2048, 7168, "bf16", 128, False),
        # decode of 16 sequences through the widest projection
        _gemm("linear_16", 16, 18432, 7168, "fp16", 32, True),
        # 64 sequences through the projection back
        _gemm("linear_64", 64, 7168, 18432, "bf16", 64, False),
        # odd sizes: columns off the tile, a last group that is short
        _gemm("linear_odd", 5, 1000, 4128, "fp16", 64, False),
        # one token's 8 experts of 256, gate and up: 248 experts without rows
        _experts("experts_token", 8, 256, 4096, 7168, "bf16", 32, True, False),
        # the down projection of a 64-token decode step, top-8 of 256
        _experts("experts_decode", 512, 256, 7168, 2048, "bf16", 128, False, False),
        # the small test layer (16 tokens, top-4): latency
        _ragged("ragged_tiny", "fwd", 64, 16, 256, 256, "fp16", "fp16", False),
        # gate and up of a prefill of 8192 tokens a GPU, 32 local experts of 256
        _ragged("ragged_prefill", "fwd", 65536, 32, 4096, 7168, "bf16", "bf16", False),
        # backward of the down projection's layer in a training step, fp32 weight gradients
        _ragged("ragged_train", "bwd", 16384, 32, 4096, 2048, "bf16", "fp32", False),
        # skewed routing with experts that get nothing, sizes off the tile
        _ragged("ragged_skew", "bwd", 5003, 48, 1000, 1160, "fp16", "fp16", True),
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["fp4", "gemm", "experts", "fwd", "bwd"])
    dtype = rng.choice(["bf16", "fp16"])
    group = rng.choice([32, 64, 128])
    e8m0 = rng.random() < 0.5
    zipf = rng.random() < 0.3
    if kind == "fp4":
        K = _log(rng, 64, 18432, 32)
        return _drop(_fp4("", _log(rng, 64, min(131072, 32 * 4096 * 7168 // K)), K, dtype, group, e8m0))
    if kind == "gemm":
        return _drop(_gemm("", _log(rng, 1, 64), _log(rng, 100, 18432), _log(rng, 128, 7168, 32), dtype, group, e8m0))
    if kind == "experts":
        E, K = _log(rng, 4, 256), _log(rng, 128, 4096, 32)
        N = _log(rng, 128, min(4096, 256 * 7168 * 2048 // (E * K)))
        return _drop(_experts("", _log(rng, 1, 1024), E, N, K, dtype, group, e8m0, zipf))
    E, N, K = _log(rng, 2, 64), _log(rng, 128, 4096, 8), _log(rng, 128, 4096, 8)
    R = _log(rng, 16, 32768 if not zipf else 8192)
    return _drop(_ragged("", kind, R, E, N, K, dtype, rng.choice([dtype, "fp32"]), zipf))


def _drop(c):
    return {k: v for k, v in c.items() if k != "name"}


def _popularity(case):
    """Share of the rows each expert is expected to get, most popular first."""
    E = case["E"]
    p = torch.arange(1, E + 1, dtype=torch.float64) ** (-_ZIPF if case["zipf"] else 0.0)
    return p / p.sum()


def work(case):
    K = case["K"]
    G = -(-K // case["group"]) if "group" in case else 0
    sb = 1 if case.get("e8m0") else 4
    if case["kind"] == "fp4":  # weights in, codes and scales out; codes and scales in, weights out
        n = case["rows"]
        return {"bytes": n * (2 * K + 2 * (K // 2 + G * sb) + 2 * K), "flops": 4 * n * K}
    if case["kind"] == "gemm":
        M, N = case["M"], case["N"]
        return {"bytes": N * (K // 2 + G * sb) + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    R, E, N = case["R"], case["E"], case["N"]
    p = _popularity(case)
    active = float((1 - (1 - p) ** R).sum())
    if case["kind"] == "experts":
        return {"bytes": active * N * (K // 2 + G * sb) + 2 * R * K + 2 * R * N + 4 * (E + 1), "flops": 2 * R * N * K}
    if case["kind"] == "fwd":
        return {"bytes": 2 * (active * N * K + R * K + R * N) + 4 * (E + 1), "flops": 2 * R * N * K}
    dw = 4 if case["dw"] == "fp32" else 2
    return {"bytes": 2 * (active * N * K + R * N) + 2 * 2 * R * K + dw * E * N * K + 4 * (E + 1), "flops": 4 * R * N * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    dt, K = _DT[case["dtype"]], case["K"]

    def normal(*shape, std=1.0, to=dt):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(to)

    st = {"case": case}
    if case["kind"] == "fp4":
        st["w"] = torch.empty((case["rows"], K), dtype=dt, device=dev)
        for i in range(0, case["rows"], 32768):
            st["w"][i:i + 32768] = normal(min(32768, case["rows"] - i), K, std=0.02)
        return st
    if case["kind"] == "gemm":
        st["x"] = normal(case["M"], K)
        st["q"], st["scale"] = _plain_quant(normal(case["N"], K, std=0.02, to=torch.float32), case["group"], case["e8m0"])
        return st
    R, E, N = case["R"], case["E"], case["N"]
    host = torch.Generator().manual_seed(int(seed) * 7919 + 18)
    p = _popularity(case)[torch.randperm(E, generator=host)]
    counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=host), minlength=E)
    st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(dev)
    st["most"] = int(counts.max())  # rows of the largest group
    if case["kind"] == "experts":
        q, s = zip(*(_plain_quant(normal(N, K, std=0.02, to=torch.float32), case["group"], case["e8m0"]) for _ in range(E)))
        st["x"], st["q"], st["scale"] = normal(R, K), torch.stack(q), torch.stack(s)
        return st
    st["w"] = torch.empty((E, N, K), dtype=dt, device=dev)
    for e in range(E):
        st["w"][e] = normal(N, K, std=0.02)
    st["x"] = normal(R, K)
    if case["kind"] == "bwd":
        st["dy"] = normal(R, N, std=0.01)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return _own(case, state) if own else _plain(case, state)


def _own(case, st):
    import fp8_block_scaled_grouped_amd as m
    if case["kind"] == "fp4":
        q, scale = m.fp4_quant_groups(st["w"], case["group"], "e8m0" if case["e8m0"] else "fp32")
        return m.fp4_dequant_groups(q, scale, case["group"], _DT[case["dtype"]])
    if case["kind"] == "gemm":
        return m.gemm_fp4_groupscale(st["x"], st["q"], st["scale"], case["group"])
    if case["kind"] == "experts":
        return m.grouped_gemm_fp4(st["x"], st["q"], st["scale"], st["offsets"], case["group"])
    if case["kind"] == "fwd":
        return m.grouped_gemm(st["x"], st["w"], st["offsets"])
    return {"dx": m.grouped_gemm_dgrad(st["dy"], st["w"], st["offsets"]),
            "dw": m.grouped_gemm_wgrad(st["dy"], st["x"], st["offsets"], out_dtype=_DT[case["dw"]])}


def _weights(q, scale, group, e8m0):
    """4-bit codes [..., N, K/2] and their scales -> fp32 weights [..., N, K]."""
    table = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float32, device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).flatten(-2)
    s = torch.ldexp(torch.ones((), device=q.device), scale.int() - 127) if e8m0 else scale
    K = v.shape[-1]
    return v.mul_(s.repeat_interleave(group, -1)[..., :K])


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


def _plain(case, st):
    dt = _DT[case["dtype"]]
    if case["kind"] == "fp4":
        q, scale = _plain_quant(st["w"], case["group"], case["e8m0"])
        return _weights(q, scale, case["group"], case["e8m0"]).to(dt)
    if case["kind"] == "gemm":
        return (st["x"].float() @ _weights(st["q"], st["scale"], case["group"], case["e8m0"]).t()).to(dt)
    off, most, R = st["offsets"].long(), st["most"], case["R"]
    if case["kind"] == "experts":
        w = _weights(st["q"], st["scale"], case["group"], case["e8m0"])
        return _ragged_rows(torch.bmm(_padded(st["x"], off, most), w.transpose(1, 2)), off, R).to(dt)
    if case["kind"] == "fwd":
        return _ragged_rows(torch.bmm(_padded(st["x"], off, most), st["w"].float().transpose(1, 2)), off, R).to(dt)
    dy = _padded(st["dy"], off, most)
    dx = _ragged_rows(torch.bmm(dy, st["w"].float()), off, R).to(dt)
    return {"dx": dx, "dw": torch.bmm(dy.transpose(1, 2), _padded(st["x"], off, most)).to(_DT[case["dw"]])}


def _plain_quant(w, group, e8m0):
    """Weights [n, K] -> (codes uint8 [n, K/2], scales); also how a checkpoint ships the weights that prepare() makes."""
    n, K = w.shape
    G = -(-K // group)
    g = torch.nn.functional.pad(w.float(), (0, G * group - K)).view(n, G, group)
    amax = g.abs().amax(-1)
    if e8m0:
        ex = torch.where(amax == 0, 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127))
        s, scale = torch.ldexp(torch.ones_like(amax), ex), (ex + 127).to(torch.uint8)
    else:
        # a quotient of tensors: by a Python number, torch multiplies by the reciprocal
        s = scale = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 6.0))
    y = g / s[..., None]
    a = y.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (m.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).view(n, G * group)[:, :K]
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), scale


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "fp4":
        return torch.cat([_exact_fp4(w, case) for w in st["w"].split(8192)]) if case["rows"] * case["K"] <= 1 << 28 else None
    if case["kind"] == "gemm":
        return st["x"].double() @ _exact_weight(st["q"], st["scale"], case).t()
    out = {k: [] for k in ("y", "dx", "dw")}
    off = st["offsets"].tolist()
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if case["kind"] == "bwd":
            dy = st["dy"][a:b].double()
            out["dx"].append(dy @ st["w"][e].double())
            out["dw"].append(dy.t() @ st["x"][a:b].double())
        elif b > a:
            w = st["w"][e].double() if case["kind"] == "fwd" else _exact_weight(st["q"][e], st["scale"][e], case)
            out["y"].append(st["x"][a:b].double() @ w.t())
    if case["kind"] == "bwd":
        return {"dx": torch.cat(out["dx"]), "dw": torch.stack(out["dw"])}
    return torch.cat(out["y"])


def _exact_weight(q, scale, case):
    """Value of code c: m/2 for the two smallest indices, else (1 + odd/2) * 2^(i/2 - 1), times the group's scale."""
    c = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    for half, codes in ((0, q % 16), (1, q // 16)):
        i = (codes % 8).double()
        e = torch.floor(i / 2)
        v = torch.where(i < 2, i / 2, (1 + (i - 2 * e) / 2) * 2.0 ** (e - 1))
        c[:, half::2] = torch.where(codes >= 8, -v, v)
    s = 2.0 ** (scale.double() - 127) if case["e8m0"] else scale.double()
    k = torch.arange(c.shape[1], device=q.device) // case["group"]
    return c * s[:, k]


def _exact_fp4(w, case):
    """Nearest of the eight levels of w over the group's scale (scale and quotient in fp32, as the format defines them)."""
    n, K = w.shape
    out = torch.empty((n, K), dtype=torch.float64, device=w.device)
    for k0 in range(0, K, case["group"]):
        x = w[:, k0:k0 + case["group"]].double()
        top = x.abs().amax(1, keepdim=True)
        safe = torch.where(top == 0, 1.0, top)
        if case["e8m0"]:
            s = 2.0 ** (torch.floor(torch.log2(safe)) - 2).clamp(-127, 127)
        else:
            s = (safe / 6).float().double()
        s = torch.where(top == 0, 1.0, s)
        y = (x / s).float().double().abs()
        best, v = torch.full_like(y, math.inf), torch.zeros_like(y)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they take the ties
            d = (y - _LEVELS[i]).abs()
            v = torch.where(d < best, _LEVELS[i], v)
            best = torch.minimum(best, d)
        out[:, k0:k0 + case["group"]] = torch.copysign(v * s, x)
    return out
