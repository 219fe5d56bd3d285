"""Cases of the dense half of a decoder layer, in 8 bits.

Four operators around the recurrence and the cached attention:

* ``norm``: the residual's addition and a root-mean-square norm, in the input's
  type or in 8 bits (read back as the values that they stand for);
* ``quant``: 8-bit floating point with a power-of-two scale for 1 x 128 values
  (activations) or 128 x 128 (weights), and the values read back;
* ``matmul``: activations times weights, both in that form, ``A W^T``;
* ``rotary``: rotary positions of queries and keys.

An 8-bit value is an E4M3 code times 2^(byte - 127): the smallest power of two,
from 2^-126 on, for which no value of the block is above 448; codes are rounded
to nearest, ties to the even code.

``run`` takes the framework's calls where ``own`` is true and elementary torch
operations in fp32 (angles in fp64) otherwise.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's norm: 256 sequences, the residual stream in bf16
        {"name": "norm_decode_256", "op": "norm", "T": 256, "C": 4096, "dt": "bf16", "add": True, "fp8": False},
        # an odd number of fp32 rows of an odd width, the first norm of a stack (nothing to add)
        {"name": "norm_odd_f32", "op": "norm", "T": 1003, "C": 1001, "dt": "f32", "add": False, "fp8": False},
        # a prompt's norm, with the projection's input in 8 bits
        {"name": "norm8_prefill_32k", "op": "norm", "T": 32768, "C": 4096, "dt": "bf16", "add": True, "fp8": True},
        # the recurrence's output of 96 heads of 128, before the output projection
        {"name": "quant_prefill_8k", "op": "quant", "T": 8192, "C": 12288, "dt": "bf16", "rows": 1},
        # a projection's weights when a model is loaded: 4 x 32 heads of 128 and 32 more rows
        {"name": "quant_weight", "op": "quant", "T": 16416, "C": 4096, "dt": "bf16", "rows": 128},
        # one user's token through that projection
        {"name": "mm_decode_1", "op": "matmul", "M": 1, "N": 16416, "K": 4096, "dt": "bf16"},
        # the step of a small stack (hidden size 512, four heads)
        {"name": "mm_small_8", "op": "matmul", "M": 8, "N": 2052, "K": 512, "dt": "bf16"},
        # the output projection of 96 heads for 256 sequences
        {"name": "mm_decode_256", "op": "matmul", "M": 256, "N": 4096, "K": 12288, "dt": "bf16"},
        # the input projection of a prompt
        {"name": "mm_prefill_8k", "op": "matmul", "M": 8192, "N": 16416, "K": 4096, "dt": "bf16"},
        # the new token of each of 256 long sequences, 96 query heads on 8 key heads, parts of the fused projection
        {"name": "rot_decode_256", "op": "rotary", "T": 256, "Hq": 96, "Hk": 8, "D": 128, "rot": 128, "pairs": "half", "scaled": True, "dt": "bf16",
         "fused": True, "spread": True},
        # small fp32 heads, the first half of each turned
        {"name": "rot_odd_f32", "op": "rotary", "T": 1003, "Hq": 6, "Hk": 2, "D": 64, "rot": 32, "pairs": "next", "scaled": False, "dt": "f32",
         "fused": False, "spread": True},
        # a long prompt
        {"name": "rot_prefill_64k", "op": "rotary", "T": 65536, "Hq": 32, "Hk": 4, "D": 128, "rot": 128, "pairs": "half", "scaled": False, "dt": "bf16",
         "fused": True, "spread": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "matmul", "matmul", "matmul", "rotary", "rotary"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm" or op == "quant":
        C = _log(rng, 16, 12288)
        if rng.random() < 0.75:
            C = -(-C // 16) * 16
        T = _log(rng, 1, max(1, min(65536, (1 << (27 if dt == "bf16" else 25)) // C)))
        if op == "norm":
            return {"op": op, "T": T, "C": C, "dt": dt, "add": rng.random() < 0.7, "fp8": rng.random() < 0.5}
        return {"op": op, "T": T, "C": C, "dt": dt, "rows": rng.choice([1, 1, 128])}
    if op == "matmul":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 16416), 16 * _log(rng, 4, 768)
        if rng.random() < 0.5:
            N = -(-N // 32) * 32
        while M * N * K > 8192 * 16416 * 4096:
            M = M // 2
        return {"op": op, "M": M, "N": N, "K": K, "dt": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    D = rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 8, 12])
    T = _log(rng, 1, max(1, min(65536, (1 << (28 if dt == "bf16" else 26)) // ((Hq + Hk) * D))))
    return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rng.choice([D, D, D // 2, D // 4]), "pairs": rng.choice(["half", "next"]),
            "scaled": rng.random() < 0.5, "dt": dt, "fused": rng.random() < 0.6, "spread": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs
def _freqs(rot, scaled):
    """Radians per position of each pair, fp64; for a long context the slow pairs are stretched and the amplitude rises with its logarithm."""
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not scaled:
        return f, 1.0
    factor, length = 16.0, 8192
    lo, hi = [rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
    keep = [1.0 - min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
    return [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0


def _rows(T, C, gen, dt):
    """Activations: normally distributed, a few channels much larger than the others."""
    x = torch.randn((T, C), device="cuda", generator=gen)
    x *= torch.exp(torch.randn((C,), device="cuda", generator=gen))
    return x.to(_DT[dt])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "norm":
        s["x"] = _rows(case["T"], case["C"], gen, case["dt"])
        s["r"] = _rows(case["T"], case["C"], gen, case["dt"]) if case["add"] else None
        s["w"] = 1.0 + 0.2 * torch.randn((case["C"],), device="cuda", generator=gen)
    elif case["op"] == "quant":
        s["x"] = _rows(case["T"], case["C"], gen, case["dt"])
    elif case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _quant(_rows(M, K, gen, "f32"), 1)
        s["w"], s["sw"] = _quant(torch.randn((N, K), device="cuda", generator=gen) * K ** -0.5, 128)
    else:
        T, D, Hq, Hk = case["T"], case["D"], case["Hq"], case["Hk"]
        x = torch.randn((T, (Hq + (2 if case["fused"] else 1) * Hk) * D), device="cuda", generator=gen).to(_DT[case["dt"]])
        q, k = x[:, :Hq * D].view(T, Hq, D), x[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["q"], s["k"] = (q, k) if case["fused"] else (q.contiguous(), k.contiguous())
        if case["spread"]:  # tokens of many sequences, some places of the batch padded
            pos = torch.randint(0, 131072, (T,), device="cuda", generator=gen)
            pos[T // 3::17] = -1
        else:  # one prompt behind a cached prefix
            pos = torch.arange(T, device="cuda") + torch.randint(0, 4096, (1,), device="cuda", generator=gen)
        s["pos"] = pos.to(torch.int32)
        f, s["amp"] = _freqs(case["rot"], case["scaled"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    return s


# ----------------------------------------------------------- plain forms
def _quant(x, rows):
    """fp32 [T, C] -> (E4M3 codes [T, C], scale bytes [ceil(T / rows), ceil(C / 128)])."""
    T, C = x.shape
    p = torch.nn.functional.pad(x, (0, -C % 128, 0, -T % rows)).view(-(-T // rows), rows, -(-C // 128), 128)
    amax = p.abs().amax((1, 3))
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), -126).clamp(min=-126)
    y = torch.ldexp(p, -e[:, None, :, None]).view(p.shape[0] * rows, -1)[:T, :C]
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, scales, rows):
    T, C = codes.shape
    s = torch.exp2(scales.float() - 127.0).repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :C]
    return codes.float() * s


def _norm_plain(s):
    x, dt = s["x"].float(), s["x"].dtype
    if s["r"] is not None:
        x = x + s["r"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * s["w"]
    out = [_values(*_quant(y, 1), 1).to(torch.bfloat16) if s["case"]["fp8"] else y.to(dt)]
    return out + ([x.to(dt)] if s["r"] is not None else [])


def _quant_plain(s):
    rows = s["case"]["rows"]
    return _values(*_quant(s["x"].float(), rows), rows).to(torch.bfloat16)


def _matmul_plain(s):
    return torch.matmul(_values(s["a"], s["sa"], 1), _values(s["w"], s["sw"], 128).t()).to(_DT[s["case"]["dt"]])


def _rotary_plain(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    ang = s["pos"].double()[:, None] * s["freq"]
    pad = (s["pos"] < 0)[:, None]
    cos = torch.where(pad, 1.0, torch.cos(ang) * s["amp"]).float()[:, None]
    sin = torch.where(pad, 0.0, torch.sin(ang) * s["amp"]).float()[:, None]

    def turn(x):
        y = x.float()
        a, b = (y[..., :half], y[..., half:rot]) if c["pairs"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
        u, v = a * cos - b * sin, a * sin + b * cos
        t = torch.cat([u, v], -1) if c["pairs"] == "half" else torch.stack([u, v], -1).flatten(-2)
        return torch.cat([t, y[..., rot:]], -1).to(x.dtype)

    return [turn(s["q"]), turn(s["k"])]


def run(s):
    if own:
        import linear_attention_recurrence_chunk_gb300 as kda
        c = s["case"]
        if s["op"] == "norm":
            if c["fp8"]:
                codes, scales, h = kda.kda_add_rmsnorm_fp8(s["x"], s["r"], s["w"], _EPS)
                y = kda.kda_fp8_values(codes, scales)
            else:
                y, h = kda.kda_add_rmsnorm(s["x"], s["r"], s["w"], _EPS)
            return [y] if h is None else [y, h]
        if s["op"] == "quant":
            codes, scales = kda.kda_fp8_quant(s["x"], c["rows"])
            return kda.kda_fp8_values(codes, scales, c["rows"])
        if s["op"] == "matmul":
            return kda.kda_fp8_matmul(s["a"], s["sa"], s["w"], s["sw"], _DT[c["dt"]])
        return list(kda.kda_rotary(s["q"], s["k"], s["pos"], s["freq"], amplitude=s["amp"], interleaved=c["pairs"] == "next"))
    return {"norm": _norm_plain, "quant": _quant_plain, "matmul": _matmul_plain, "rotary": _rotary_plain}[s["op"]](s)


# -------------------------------------------------------------- work and truth
def work(case):
    eb = 2 if case.get("dt") == "bf16" else 4
    if case["op"] == "norm":
        n, groups = case["T"] * case["C"], case["T"] * -(-case["C"] // 128)
        y = 2 * (n + groups) + 2 * n if case["fp8"] else n * eb  # 8 bits written and read back, the values written
        return {"bytes": n * eb * (3 if case["add"] else 1) + y + 4 * case["C"], "flops": 0}
    if case["op"] == "quant":
        n, groups = case["T"] * case["C"], -(-case["T"] // case["rows"]) * -(-case["C"] // 128)
        return {"bytes": n * eb + 2 * (n + groups) + 2 * n, "flops": 0}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + -(-K // 128) * (M + -(-N // 128)) + M * N * eb, "flops": 2 * M * N * K}
    return {"bytes": 2 * case["T"] * (case["Hq"] + case["Hk"]) * case["D"] * eb + 4 * case["T"] + 4 * case["rot"], "flops": 0}


def _truth_round(x, rows):
    """What 8 bits hold of x, in fp64: each block on the grid of its scale."""
    x = x.double()
    T, C = x.shape
    p = torch.zeros((T + -T % rows, C + -C % 128), dtype=torch.float64, device=x.device)
    p[:T, :C] = x
    b = p.view(-1, rows, p.shape[1] // 128, 128).transpose(1, 2).flatten(2)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 10  # 448 * 2^e is below amax; then the first that is not
    for _ in range(4):
        e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    unit = torch.exp2(torch.where(amax > 0, e, -126.0).clamp(min=-126.0))
    y = b.abs() / unit
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    v = torch.sign(b) * torch.round(y / step) * step * unit
    return v.view(-1, p.shape[1] // 128, rows, 128).transpose(1, 2).reshape(p.shape)[:T, :C]


def _truth_code(codes, scales, rows):
    """The values of codes, from their bits."""
    c = codes.view(torch.uint8).long()
    exp, man = c >> 3 & 15, c & 7
    v = torch.where(exp > 0, (8 + man).double() * torch.exp2(exp.double() - 10), man.double() * 2.0 ** -9)
    v = torch.where(c >= 128, -v, v)
    i, j = torch.arange(c.shape[0], device=c.device) // rows, torch.arange(c.shape[1], device=c.device) // 128
    return v * torch.exp2(scales.double() - 127)[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = h + s["r"].double()
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["C"] + _EPS) * s["w"].double()
        return [_truth_round(y, 1) if case["fp8"] else y] + ([h] if s["r"] is not None else [])
    if case["op"] == "quant":
        return _truth_round(s["x"], case["rows"])
    if case["op"] == "matmul":
        return torch.einsum("mk,nk->mn", _truth_code(s["a"], s["sa"], 1), _truth_code(s["w"], s["sw"], 128))
    ang = s["pos"].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.full_like(ang, s["amp"]), ang)
    turn = torch.where((s["pos"] < 0)[:, None, None], torch.ones_like(turn), turn)
    rot, got = case["rot"], []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        if case["pairs"] == "half":
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            y[..., :rot] = torch.view_as_real(torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        got.append(y)
    return got
