"""Cases of the microscaled (MX) operators: what is measured of them and what they compute.

Operators of token_dispatch_moe_b200 that the cases call:
  moe_add_rmsnorm         residual addition and root-mean-square norm, with an MX output
  moe_mx_quantize, moe_mx_dequantize
                          bf16 rows to microscaled 8- or 4-bit rows, and back
  moe_expert_gate_up_mx   the experts' gate and up products on MX operands, SwiGLU, MX output
  moe_expert_down_mx      the experts' down product on MX operands

An MX row of K values: blocks of 32 values share one power of two (a byte b
stands for 2^(b - 127)); the values are e4m3 (a byte) or e2m1 (four bits, the
even column in the low half).  Rows are padded with zeros to a multiple of 128
values, scale rows to a multiple of 16 bytes.  A block's scale is the smallest
power of two with which no value of the block saturates (2^-127 at least);
values round to nearest, ties to even.

``run`` computes the operators from elementary torch operations where ``own``
is false, and calls the framework where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, E2M1 = 0, 1            # formats
SWIGLU, SWIGLU_OAI = 0, 1    # activations


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token in front of a gpt-oss layer: the latency of the norm
        dict(name="norm_token", kind="norm", T=1, d=2880, residual=True, fmt=E4M3),
        # a prompt batch at the qwen3 width, 4-bit activations
        dict(name="norm_16384x2048_e2m1", kind="norm", T=16384, d=2048, residual=True, fmt=E2M1),
        # the largest batch of the router's workloads
        dict(name="norm_65536x7168", kind="norm", T=65536, d=7168, residual=True, fmt=E4M3),
        # a gate or up matrix of all gpt-oss experts, converted from and back to bf16
        dict(name="mx_experts_e2m1", kind="mx", rows=128 * 2880, K=2880, fmt=E2M1),
        # an odd batch of activations whose width ends inside a block
        dict(name="mx_odd_e4m3", kind="mx", rows=1023, K=2056, fmt=E4M3),
        # one token decoded by gpt-oss experts: four experts' weights are the work
        dict(name="gate_up_token", kind="gate_up", T=1, k=4, E=128, d=2880, F=2880, act=SWIGLU_OAI, bias=True, fmt=E4M3, wfmt=E2M1, hot=0),
        # a decode batch: nearly every expert is read for two or three rows
        dict(name="gate_up_batch", kind="gate_up", T=64, k=4, E=128, d=2880, F=2880, act=SWIGLU_OAI, bias=True, fmt=E4M3, wfmt=E2M1, hot=0),
        # a prompt batch through the qwen3 experts, one expert in demand, 8-bit weights
        dict(name="gate_up_qwen3", kind="gate_up", T=16384, k=8, E=128, d=2048, F=768, act=SWIGLU, bias=False, fmt=E4M3, wfmt=E4M3, hot=1),
        # a prompt batch through the gpt-oss experts
        dict(name="gate_up_gptoss", kind="gate_up", T=32768, k=4, E=128, d=2880, F=2880, act=SWIGLU_OAI, bias=True, fmt=E4M3, wfmt=E2M1, hot=0),
        # the down product of one decoded token
        dict(name="down_token", kind="down", T=1, k=4, E=128, d=2880, F=2880, bias=True, fmt=E4M3, wfmt=E2M1, hot=0),
        # a few hundred tokens: ragged blocks of some tens of rows
        dict(name="down_ragged", kind="down", T=509, k=4, E=128, d=2880, F=2880, bias=True, fmt=E4M3, wfmt=E2M1, hot=1),
        # the down product of a prompt batch
        dict(name="down_gptoss", kind="down", T=32768, k=4, E=128, d=2880, F=2880, bias=True, fmt=E4M3, wfmt=E2M1, hot=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "mx", "gate_up", "down", "gate_up", "down"])
    fmt = rng.choice([E4M3, E4M3, E2M1])
    if kind == "norm":
        d = 8 * _log(rng, 4, 1024)
        T = _log(rng, 1, min(65536, 65536 * 7168 // d))
        return dict(kind=kind, T=T, d=d, residual=rng.random() < 0.75, fmt=fmt)
    if kind == "mx":
        K = 8 * _log(rng, 4, 1024)
        return dict(kind=kind, rows=_log(rng, 1, min(400000, 128 * 2880 * 2880 // K)), K=K, fmt=fmt)
    c = dict(kind=kind, act=rng.choice([SWIGLU, SWIGLU_OAI]), bias=rng.random() < 0.5, fmt=fmt, wfmt=rng.choice([E2M1, E2M1, E4M3]), hot=rng.choice([0, 0, 1]))
    if kind == "down":
        del c["act"]
    most = 128 * 2880 * 2880
    c["d"] = 8 * _log(rng, 8, 900)
    c["F"] = 8 * _log(rng, 8, 512)
    c["E"] = _log(rng, 2, min(256, max(2, most // (c["d"] * c["F"]))))
    c["k"] = rng.randint(1, min(8, c["E"]))
    # the padded blocks of the plain form count: a hot expert makes them longer
    rows = 131072 * 2880 * 2880 // (c["d"] * c["F"]) // (4 if c["hot"] else 1)
    c["T"] = _log(rng, 1, max(1, min(32768, rows // c["k"])))
    return c


# ----------------------------------------------------------------- MX rows --
def _up(n, m):
    return (n + m - 1) // m * m


def _scale_pitch(K):
    return _up(_up(K, 128) // 32, 16)


_HALVES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _power(e):
    """2^e in fp32 for integers e in [-126, 127], exactly."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _mx_blocks(v, fmt):
    """(scaled values [rows, Kp] fp32, exponents [rows, Kp/32] int32) of bf16 or fp32 rows."""
    rows, K = v.shape
    v = torch.nn.functional.pad(v.float(), (0, _up(K, 128) - K)).view(rows, -1, 32)
    m, e = torch.frexp(v.abs().amax(2))  # amax = m * 2^e with 0.5 <= m < 1
    # the largest values are 448 = 0.875 * 2^9 and 6 = 0.75 * 2^3
    top, at = (0.875, 9) if fmt == E4M3 else (0.75, 3)
    s = torch.where(m == 0, torch.full_like(e, -127), e - at + (m > top).to(torch.int32)).clamp(-127, 127)
    return (v * _power(-s).unsqueeze(2)).view(rows, -1), s


def _e2m1_code(a):
    """Codes 0..7 of non-negative scaled values: nearest, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c


def _quantize(v, fmt):
    """MX rows in the framework's layout: (q uint8 [rows, row bytes], scales uint8 [rows, pitch])."""
    scaled, s = _mx_blocks(v, fmt)
    if fmt == E4M3:
        q = scaled.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        code = _e2m1_code(scaled.abs()) | (torch.signbit(scaled).to(torch.uint8) << 3)
        q = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = torch.zeros((v.shape[0], _scale_pitch(v.shape[1])), dtype=torch.uint8, device=v.device)
    scales[:, :s.shape[1]] = (s + 127).to(torch.uint8)
    return q, scales


def _elements(q, fmt):
    """The element values [..., Kp] fp32 of rows of codes."""
    if fmt == E4M3:
        return q.view(torch.float8_e4m3fn).float()
    table = torch.tensor(_HALVES + [-x for x in _HALVES], dtype=torch.float32, device=q.device)
    pairs = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    return table[pairs.int()]


def _dequantize(q, scales, fmt):
    """The values [..., Kp] fp32 that MX rows stand for."""
    v = _elements(q, fmt)
    n = v.shape[-1] // 32
    two = torch.ldexp(torch.ones((), device=q.device), torch.arange(-127, 129, device=q.device).double()).float()
    return (v.unflatten(-1, (n, 32)) * two[scales[..., :n].int()].unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ inputs --
def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed % 1000003) + k)
    return g


def _randn(shape, seed, k, std=1.0):
    return torch.randn(shape, generator=_gen(seed, k), device=DEV).mul_(std)


def _activations(rows, width, seed, k):
    """Hidden rows: normal, of different size from row to row, a few channels far larger."""
    v = _randn((rows, width), seed, k)
    v *= torch.exp(0.5 * _randn((rows, 1), seed, k + 1))
    loud = torch.randperm(width, generator=_gen(seed, k + 2), device=DEV)[:max(1, width // 256)]
    v[:, loud] *= 12.0
    return v.to(torch.bfloat16)


def _weights(E, rows, K, fmt, seed, k):
    """Every expert's matrix [rows, K] ~ N(0, 1/K) as MX rows, expert by expert."""
    row = _up(K, 128) // (1 if fmt == E4M3 else 2)
    q = torch.empty((E, rows, row), dtype=torch.uint8, device=DEV)
    s = torch.empty((E, rows, _scale_pitch(K)), dtype=torch.uint8, device=DEV)
    g = _gen(seed, k)
    per = max(1, (1 << 26) // (rows * K))
    for e in range(0, E, per):
        n = min(per, E - e)
        w = torch.randn((n * rows, K), generator=g, device=DEV).mul_(K ** -0.5)
        a, b = _quantize(w.to(torch.bfloat16), fmt)
        q[e:e + n], s[e:e + n] = a.view(n, rows, row), b.view(n, rows, -1)
    return q, s


def _routing(c, seed):
    """Block offsets of T tokens that pick k distinct experts each (hot: one expert is liked more)."""
    logits = _randn((c["T"], c["E"]), seed, 1)
    if c["hot"]:
        logits[:, seed % c["E"]] += 1.0
    ids = logits.topk(c["k"], dim=1).indices.flatten()
    counts = torch.bincount(ids, minlength=c["E"])
    offsets = torch.zeros((c["E"] + 1,), dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, counts


def prepare(case, seed):
    c = dict(case)
    if c["kind"] == "norm":
        T, d = c["T"], c["d"]
        c["x"] = _activations(T, d, seed, 2)
        c["r"] = _randn((T, d), seed, 6, 2.0).to(torch.bfloat16) if c["residual"] else None
        c["gain"] = (1.0 + 0.2 * _randn((d,), seed, 7)).to(torch.bfloat16)
        c["eps"] = 1e-5
        c["r_out"] = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
        c["y"] = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
        c["out"] = _mx_out(T, d, c["fmt"])
        return c
    if c["kind"] == "mx":
        c["x"] = _activations(c["rows"], c["K"], seed, 2)
        c["out"] = _mx_out(c["rows"], c["K"], c["fmt"])
        c["back"] = torch.empty((c["rows"], c["K"]), dtype=torch.bfloat16, device=DEV)
        return c
    E, d, F, N = c["E"], c["d"], c["F"], c["T"] * c["k"]
    c["offsets"], counts = _routing(c, seed)
    c["active"] = counts.nonzero().flatten()
    c["longest"] = int(counts.max())
    c["N"] = N
    c["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    c["x"] = _quantize(_activations(N, d if c["kind"] == "gate_up" else F, seed, 2), c["fmt"])
    if c["kind"] == "gate_up":
        c["w1"] = _weights(E, F, d, c["wfmt"], seed, 20)
        c["w3"] = _weights(E, F, d, c["wfmt"], seed, 21)
        c["b1"] = _randn((E, F), seed, 22, 0.5) if c["bias"] else None
        c["b3"] = _randn((E, F), seed, 23, 0.5) if c["bias"] else None
        c["out"] = _mx_out(N, F, c["fmt"])
    else:
        c["w2"] = _weights(E, d, F, c["wfmt"], seed, 24)
        c["b2"] = _randn((E, d), seed, 25, 0.5) if c["bias"] else None
        c["y"] = torch.empty((N, d), dtype=torch.bfloat16, device=DEV)
    return c


def _mx_out(rows, K, fmt):
    row = _up(K, 128) // (1 if fmt == E4M3 else 2)
    return (torch.empty((rows, row), dtype=torch.uint8, device=DEV),
            torch.empty((rows, _scale_pitch(K)), dtype=torch.uint8, device=DEV))


# --------------------------------------------------------------- the passes --
def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "mx": _plain_mx, "gate_up": _plain_gate_up, "down": _plain_down}[state["kind"]](state)


def _run_own(c):
    import token_dispatch_moe_b200 as moe
    if c["kind"] == "norm":
        mx = moe.MxRows(*c["out"], c["d"], c["fmt"])
        moe.moe_add_rmsnorm(c["x"], c["r"], c["gain"], c["eps"], c["r_out"] if c["residual"] else None, c["y"], mx)
        out = {"y": c["y"], "mx": _typed(c["out"], c["d"], c["fmt"], moe)}
        return {**out, "residual": c["r_out"]} if c["residual"] else out
    if c["kind"] == "mx":
        mx = moe.MxRows(*c["out"], c["K"], c["fmt"])
        moe.moe_mx_quantize(c["x"], mx)
        moe.moe_mx_dequantize(mx, c["back"])
        return {"values": c["back"], "scales": c["out"][1][:, :_up(c["K"], 32) // 32]}
    x = moe.MxRows(*c["x"], c["d"] if c["kind"] == "gate_up" else c["F"], c["fmt"])
    if c["kind"] == "gate_up":
        h = moe.MxRows(*c["out"], c["F"], c["fmt"])
        w1, w3 = moe.MxRows(*c["w1"], c["d"], c["wfmt"]), moe.MxRows(*c["w3"], c["d"], c["wfmt"])
        moe.moe_expert_gate_up_mx(x, c["offsets"], w1, w3, h, c["b1"], c["b3"], c["act"], c["status"])
        return _typed(c["out"], c["F"], c["fmt"], moe)
    moe.moe_expert_down_mx(x, c["offsets"], moe.MxRows(*c["w2"], c["F"], c["wfmt"]), c["y"], c["b2"], c["status"])
    return c["y"]


def _typed(out, K, fmt, moe):
    """MX rows as values: e4m3 bytes and their scales as they are, typed; 4-bit values as bf16."""
    if fmt == E4M3:
        return {"elements": out[0].view(torch.float8_e4m3fn)[:, :K], "scales": out[1].view(torch.float8_e8m0fnu)[:, :_up(K, 32) // 32]}
    values = torch.empty((out[0].shape[0], K), dtype=torch.bfloat16, device=out[0].device)
    moe.moe_mx_dequantize(moe.MxRows(*out, K, fmt), values)
    return {"values": values}


def _plain_typed(v, fmt):
    """What _typed returns of the MX rows of v."""
    K = v.shape[1]
    scaled, s = _mx_blocks(v, fmt)
    if fmt == E4M3:
        return {"elements": scaled.to(torch.float8_e4m3fn)[:, :K], "scales": (s + 127).to(torch.uint8)[:, :_up(K, 32) // 32].contiguous().view(torch.float8_e8m0fnu)}
    q, scales = _quantize(v, fmt)
    return {"values": _dequantize(q, scales, fmt)[:, :K].to(torch.bfloat16)}


def _plain_norm(c):
    r = c["x"]
    if c["residual"]:
        r = (c["x"].float() + c["r"].float()).to(torch.bfloat16)
    f = r.float()
    f = f * torch.rsqrt((f * f).mean(1, keepdim=True) + c["eps"])
    y = (f * c["gain"].float()).to(torch.bfloat16)
    out = {"y": y, "mx": _plain_typed(y, c["fmt"])}
    return {**out, "residual": r} if c["residual"] else out


def _plain_mx(c):
    q, scales = _quantize(c["x"], c["fmt"])
    v = _dequantize(q, scales, c["fmt"])[:, :c["K"]]
    return {"values": v.to(torch.bfloat16), "scales": scales[:, :_up(c["K"], 32) // 32]}


def _blocks(c):
    """Row of every (active expert, place), and which places hold a row."""
    first = c["offsets"][c["active"]].long()
    last = c["offsets"][c["active"] + 1].long()
    at = first.unsqueeze(1) + torch.arange(c["longest"], device=DEV)
    there = at < last.unsqueeze(1)
    return at.clamp(max=c["N"] - 1), there


def _products(c, x, w, b):
    """x [experts, places, Kp] times each active expert's matrix, plus its bias."""
    y = torch.bmm(x, _dequantize(w[0][c["active"]], w[1][c["active"]], c["wfmt"]).transpose(1, 2))
    return y if b is None else y.add_(b[c["active"]].unsqueeze(1))


def _activate(g, u, act):
    if act == SWIGLU:
        return g * torch.sigmoid(g) * u
    g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
    return g * torch.sigmoid(1.702 * g) * (u + 1.0)


def _plain_gate_up(c):
    at, there = _blocks(c)
    x = _dequantize(*c["x"], c["fmt"])[at]
    h = _activate(_products(c, x, c["w1"], c["b1"]), _products(c, x, c["w3"], c["b3"]), c["act"])
    # the rows of the blocks in order are the rows of the result
    return _plain_typed(h[there], c["fmt"])


def _plain_down(c):
    at, there = _blocks(c)
    return _products(c, _dequantize(*c["x"], c["fmt"])[at], c["w2"], c["b2"])[there].to(torch.bfloat16)


# --------------------------------------------------------------------- work --
def _mx_bytes(rows, K, fmt):
    return rows * K * ((1.0 if fmt == E4M3 else 0.5) + 1.0 / 32)


def work(case):
    c = case
    if c["kind"] == "norm":
        n = c["T"] * c["d"]
        return {"bytes": n * (8 if c["residual"] else 4) + 2 * c["d"] + _mx_bytes(c["T"], c["d"], c["fmt"]), "flops": 8 * n}
    if c["kind"] == "mx":  # to the MX rows, and from them back
        return {"bytes": 4 * c["rows"] * c["K"] + 2 * _mx_bytes(c["rows"], c["K"], c["fmt"]), "flops": 4 * c["rows"] * c["K"]}
    E, d, F, N = c["E"], c["d"], c["F"], c["T"] * c["k"]
    used = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])  # experts that some row is for, on average
    if c["kind"] == "gate_up":
        b = _mx_bytes(N, d, c["fmt"]) + 2 * _mx_bytes(used * F, d, c["wfmt"]) + _mx_bytes(N, F, c["fmt"])
        return {"bytes": b + (8 * used * F if c["bias"] else 0), "flops": 4.0 * N * d * F}
    b = _mx_bytes(N, F, c["fmt"]) + _mx_bytes(used * d, F, c["wfmt"]) + 2 * N * d
    return {"bytes": b + (4 * used * d if c["bias"] else 0), "flops": 2.0 * N * d * F}


# -------------------------------------------------------------------- exact --
def _double_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decode64(q, scales, fmt):
    """The values of MX rows, from the fields of their codes."""
    if fmt == E2M1:
        q = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    mant, bias, sign = (3, 7, 7) if fmt == E4M3 else (1, 1, 3)
    q = q.to(torch.int64)
    e, m = (q >> mant) & ((1 << (sign - mant)) - 1), (q & ((1 << mant) - 1)).double() / (1 << mant)
    v = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * _double_power(e - bias))
    v = torch.where((q >> sign) & 1 == 1, -v, v)
    s = _double_power(scales[..., :v.shape[-1] // 32].to(torch.int64) - 127)
    return v * s.repeat_interleave(32, dim=-1)


def _encode64(v, fmt):
    """(element values, powers of two) of rows in 64 bits."""
    rows, K = v.shape
    largest, least, mant = (448.0, -6, 3) if fmt == E4M3 else (6.0, 0, 1)
    exps = torch.arange(-127, 128, device=v.device)
    full = torch.zeros((rows, _up(K, 32)), dtype=torch.float64, device=v.device)
    full[:, :K] = v
    full = full.view(rows, -1, 32)
    s = torch.searchsorted(largest * _double_power(exps), full.abs().amax(2).contiguous()).clamp(max=254) - 127
    power = _double_power(s)
    x = full / power.unsqueeze(2)
    e = torch.frexp(x)[1].to(torch.int64) - 1
    step = _double_power(torch.where(x == 0, torch.zeros_like(e), e).clamp(min=least) - mant)
    x = torch.round(x / step) * step
    return x.view(rows, -1)[:, :K], power


def _exact_typed(v, fmt):
    """The rows' elements and scales, or 4-bit rows' values, a slice of rows at a time."""
    parts = [_encode64(p, fmt) for p in v.split(max(1, (1 << 27) // v.shape[1]))]
    if fmt == E4M3:
        return {"elements": torch.cat([x for x, _ in parts]), "scales": torch.cat([p for _, p in parts])}
    return {"values": torch.cat([x * p.repeat_interleave(32, dim=1)[:, :x.shape[1]] for x, p in parts])}


def exact(case, seed):
    c = prepare(case, seed)
    if c["kind"] == "norm":
        ys, rs = [], []
        per = max(1, (1 << 26) // c["d"])
        for i in range(0, c["T"], per):
            f = c["x"][i:i + per].double()
            if c["residual"]:
                f = (f + c["r"][i:i + per].double()).to(torch.bfloat16).double()  # the sum is stored in bf16
                rs.append(f)
            mean = f.square().sum(1, keepdim=True) / c["d"]
            # y is defined as rounded to bf16, and the MX rows are those of the rounded y
            ys.append((f / torch.sqrt(mean + c["eps"]) * c["gain"].double()).to(torch.bfloat16))
        y = torch.cat(ys)
        parts = [_exact_typed(p.double(), c["fmt"]) for p in y.split(per)]
        out = {"y": y.double(), "mx": {k: torch.cat([p[k] for p in parts]) for k in parts[0]}}
        return {**out, "residual": torch.cat(rs)} if c["residual"] else out
    if c["kind"] == "mx":
        values = []
        for p in c["x"].split(max(1, (1 << 26) // c["K"])):
            v, power = _encode64(p.double(), c["fmt"])
            values.append((v * power.repeat_interleave(32, dim=1)[:, :c["K"]]).to(torch.bfloat16))
        return {"values": torch.cat(values), "scales": None}
    ends = c["offsets"].tolist()
    rows = torch.empty((c["N"], c["F"] if c["kind"] == "gate_up" else c["d"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        x = _decode64(c["x"][0][a:b], c["x"][1][a:b], c["fmt"])

        def product(w, bias):
            y = x @ _decode64(w[0][e], w[1][e], c["wfmt"]).T
            return y if bias is None else y + bias[e].double()

        if c["kind"] == "down":
            rows[a:b] = product(c["w2"], c["b2"])
            continue
        g, u = product(c["w1"], c["b1"]), product(c["w3"], c["b3"])
        if c["act"] == SWIGLU_OAI:
            g, u = torch.clamp(g, max=7.0), torch.clamp(u, -7.0, 7.0)
            rows[a:b] = g / (1.0 + torch.exp(-1.702 * g)) * (u + 1.0)
        else:
            rows[a:b] = g / (1.0 + torch.exp(-g)) * u
    return rows if c["kind"] == "down" else _exact_typed(rows, c["fmt"])
