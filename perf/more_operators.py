"""Cases of the operators around a projection: the norm in front of it, the low-rank adapters beside
it and the rotary positions behind it, each in its plain form (elementary torch operations in 32 bits)
and, where ``own`` is true, through the library's entry points.

  norm      h = x + r (stored as r is), y = h / sqrt(mean h^2 + eps) * w; y as BF16, as MXFP8 (E4M3
            codes and a power of two per 32) or as INT8 codes with a scale per row
  adapters  C = base + scale[a] * B_a (A_a x), a the adapter of each token (-1: none)
  rotary    pairs of each head's values turned by position * frequency
"""
import math

import torch

own = False

EPS = 1e-5


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence's token in front of the gate and up projections (decode: latency)
        dict(name="norm token", op="norm", rows=1, K=4096, x="bf16", r="bf16", y=False, q="mxfp8",
             pad=0),
        # a decode batch of a wider model; the BF16 rows are for the adapters
        dict(name="norm batch 64", op="norm", rows=64, K=7168, x="bf16", r="bf16", y=True, q="mxfp8",
             pad=0),
        # a ragged prompt out of a wider tensor, FP32 sums of an INT8 product, INT8 out
        dict(name="norm ragged 333", op="norm", rows=333, K=1040, x="f32", r="f32", y=False,
             q="int8", pad=48),
        # a long prompt: residual, BF16 rows and their MXFP8 codes
        dict(name="norm prompt 8192", op="norm", rows=8192, K=4096, x="bf16", r="bf16", y=True,
             q="mxfp8", pad=0),
        # one token of one request with an adapter
        dict(name="adapters token", op="adapters", M=1, N=4096, K=4096, L=4, R=16, mixed=False,
             runs=False, c="bf16", pad=0),
        # a decode batch, each token of a request of its own, adapters of different ranks
        dict(name="adapters batch 64", op="adapters", M=64, N=14336, K=4096, L=32, R=64, mixed=True,
             runs=False, c="bf16", pad=0),
        # chunks of a few requests on a block of odd width, FP32 results
        dict(name="adapters ragged 777", op="adapters", M=777, N=1001, K=1040, L=5, R=24, mixed=True,
             runs=True, c="f32", pad=40),
        # long prompts of a few requests through an up projection
        dict(name="adapters prompt 4096", op="adapters", M=4096, N=14336, K=4096, L=8, R=64,
             mixed=False, runs=True, c="bf16", pad=0),
        # the queries and keys of one token, far into its context
        dict(name="rotary token", op="rotary", T=1, heads=40, D=128, rot=128, layout="half",
             type="bf16", far=1 << 17, factor=1.0, pad=0),
        # a decode batch, half of each head in interleaved pairs
        dict(name="rotary batch 256", op="rotary", T=256, heads=36, D=128, rot=64,
             layout="interleaved", type="f16", far=1 << 15, factor=1.0, pad=1024),
        # a ragged prompt with odd heads in FP32, positions scaled for a long context
        dict(name="rotary ragged 1111", op="rotary", T=1111, heads=5, D=80, rot=40, layout="half",
             type="f32", far=1 << 20, factor=8.0, pad=7),
        # a long prompt: the query and key heads of rows that hold the values too
        dict(name="rotary prompt 16384", op="rotary", T=16384, heads=40, D=128, rot=128,
             layout="half", type="bf16", far=1 << 17, factor=4.0, pad=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "adapters", "rotary"])
    if op == "norm":
        K = 32 * _log_int(rng, 2, 512)
        return dict(op=op, rows=_log_int(rng, 1, min(16384, 8192 * 4096 // K)), K=K,
                    x=rng.choice(["bf16", "bf16", "f32"]), r=rng.choice(["bf16", "f32", "none"]),
                    y=rng.random() < 0.5, q=rng.choice(["mxfp8", "mxfp8", "int8"]),
                    pad=8 * rng.choice([0, 0, 1, 13]))
    if op == "adapters":
        K, N = 8 * _log_int(rng, 8, 1792), _log_int(rng, 16, 14336)
        R, L = rng.choice([8, 16, 24, 32, 64, 128]), _log_int(rng, 1, 64)
        cap = 4096 * (14336 + 4096) * 8 * 64 // ((N + K) * L * R)
        return dict(op=op, M=_log_int(rng, 1, max(1, min(8192, cap))), N=N, K=K, L=L, R=R,
                    mixed=rng.random() < 0.5, runs=rng.random() < 0.6,
                    c=rng.choice(["bf16", "bf16", "f32"]), pad=8 * rng.choice([0, 0, 1, 5]))
    D = rng.choice([64, 72, 80, 96, 128, 192, 256])
    heads = _log_int(rng, 1, 64)
    kind = rng.choice(["bf16", "f16", "f32"])
    cap = 16384 * 40 * 128 * 2 // (heads * D * (4 if kind == "f32" else 2))
    return dict(op=op, T=_log_int(rng, 1, min(32768, cap)), heads=heads, D=D,
                rot=rng.choice([D, D, D // 2, D // 4 * 2 - 2]),
                layout=rng.choice(["half", "interleaved"]), type=kind,
                far=_log_int(rng, 1 << 10, 1 << 21), factor=rng.choice([1.0, 4.0, 32.0]),
                pad=rng.choice([0, 0, 3, 64]))


# ----------------------------------------------------------------------------- the inputs
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _rows(rows, K, pad, dtype, gen):
    """Rows of different magnitude with a few loud channels, out of a wider tensor where pad > 0."""
    wide = torch.randn((rows, K + pad), generator=gen, device="cuda")
    wide *= torch.exp2(torch.randint(-2, 3, (rows, 1), generator=gen, device="cuda").float())
    loud = torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")
    wide[:, loud] *= 12.0
    return wide.to(dtype)[:, :K]


def _prepare_norm(s, gen):
    rows, K = s["rows"], s["K"]
    x = _rows(rows, K, s["pad"], _DTYPES[s["x"]], gen)
    r = out = None
    if s["r"] != "none":
        r = _rows(rows, K, 0, _DTYPES[s["r"]], gen)
        out = torch.empty_like(r)
    w = (1.0 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(torch.bfloat16)
    y = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda") if s["y"] else None
    if s["q"] == "mxfp8":
        codes = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
        scale = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    else:
        codes = torch.empty((rows, K), dtype=torch.int8, device="cuda")
        scale = torch.empty(rows, device="cuda")
        s["values"] = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    s.update(X=x, R=r, R_out=out, W=w, Y=y, codes=codes, scale=scale)


def _prepare_adapters(s, gen):
    M, N, K, L, R = (s[k] for k in ("M", "N", "K", "L", "R"))
    x = _rows(M, K, s["pad"], torch.bfloat16, gen)
    a = (torch.randn((L, R, K), generator=gen, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
    b = (torch.randn((L, N, R), generator=gen, device="cuda") / math.sqrt(R)).to(torch.bfloat16)
    scales = torch.rand(L, generator=gen, device="cuda") * 0.5 + 0.25
    ranks = torch.full((L,), R, dtype=torch.int32, device="cuda")
    if s["mixed"]:
        ranks = torch.randint(1, R + 1, (L,), generator=gen, device="cuda", dtype=torch.int32)
        ranks[::2] = max(1, R // 2)
        ranks[0] = R
    pick = torch.randint(0, L, (M,), generator=gen, device="cuda", dtype=torch.int32)
    none = torch.rand(M, generator=gen, device="cuda") < 0.1
    if M == 1:
        none[:] = False
    pick = torch.where(none, torch.full_like(pick, -1), pick)
    if s["runs"]:  # the tokens of a request stand together
        starts = torch.rand(M, generator=gen, device="cuda") < 8.0 / M
        starts[0] = True
        pick = pick[torch.cummax(torch.where(starts, torch.arange(M, device="cuda"), 0), 0).values]
    base = 2.0 * torch.randn((M, N), generator=gen, device="cuda")
    base = base.to(_DTYPES[s["c"]])
    s.update(X=x, A=a, B=b, scales=scales, ranks=ranks, ids=pick.contiguous(), base=base,
             C=torch.empty_like(base))


def _prepare_rotary(s, gen):
    T, n = s["T"], s["heads"] * s["D"]
    wide = torch.empty((T, n + s["pad"]), dtype=_DTYPES[s["type"]], device="cuda")
    for i in range(0, T, 4096):
        wide[i:i + 4096] = torch.randn((min(4096, T - i), n + s["pad"]), generator=gen, device="cuda")
    first = torch.randint(0, s["far"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    if T > 512:  # a prompt's positions follow one another
        first = first[0] + torch.arange(T, device="cuda", dtype=torch.int32)
    half = torch.arange(s["rot"] // 2, dtype=torch.float64, device="cuda")
    base = 10000.0 * s["factor"] ** (s["rot"] / max(1, s["rot"] - 2))
    freqs = torch.pow(torch.full_like(half, base), -half * 2 / s["rot"])
    s.update(X=wide[:, :n], positions=first, freqs=freqs,
             attention=0.1 * math.log(s["factor"]) + 1.0,
             Y=torch.empty((T, n), dtype=wide.dtype, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    {"norm": _prepare_norm, "adapters": _prepare_adapters, "rotary": _prepare_rotary}[s["op"]](s, gen)
    return s


# ----------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    h, got = s["X"].float(), {}
    if s["R"] is not None:
        got["h"] = (h + s["R"].float()).to(s["R"].dtype)
        h = got["h"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["W"].float()
    if s["y"]:
        got["y"] = y.to(torch.bfloat16)
    if s["q"] == "mxfp8":
        g = y.view(s["rows"], -1, 32)
        top = g.abs().amax(dim=2, keepdim=True)
        e = (torch.frexp(top).exponent - 9).clamp(-127, 127)
        e = torch.where(top > 0, e, torch.full_like(e, -127))
        codes = torch.ldexp(g, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        got["codes"] = codes.view(s["rows"], -1)
        got["scale"] = (e[:, :, 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        top = y.abs().amax(dim=1)
        got["scale"] = top / 127.0
        codes = torch.round(y * (127.0 / top)[:, None])
        got["values"] = (codes * got["scale"][:, None]).to(torch.bfloat16)
    return got


def _plain_adapters(s):
    """All adapters' products, with the rows that are not an adapter's own taken out between."""
    L, R, M = s["L"], s["R"], s["M"]
    there = torch.arange(R, device="cuda") < s["ranks"][:, None]
    t = (s["X"].float() @ s["A"].float().view(L * R, -1).t()).view(M, L, R)
    mine = s["ids"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32)
    t = torch.where(mine[:, :, None] & there, t * s["scales"][:, None], torch.zeros_like(t))
    b = s["B"].float().transpose(1, 2)
    b = torch.where(there[:, :, None], b, torch.zeros_like(b)).reshape(L * R, -1)
    return (s["base"].float() + t.view(M, L * R) @ b).to(s["C"].dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos = (angle.cos() * s["attention"]).float()[:, None, :]
    sin = (angle.sin() * s["attention"]).float()[:, None, :]
    x = s["X"].float().reshape(s["T"], s["heads"], s["D"])
    n = s["rot"]
    out = x.clone()
    if s["layout"] == "half":
        a, b = x[:, :, :n // 2], x[:, :, n // 2:n]
        out[:, :, :n // 2], out[:, :, n // 2:n] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[:, :, 0:n:2], x[:, :, 1:n:2]
        out[:, :, 0:n:2], out[:, :, 1:n:2] = a * cos - b * sin, b * cos + a * sin
    return out.view(s["T"], -1).to(s["Y"].dtype)


# ----------------------------------------------------------------------------- the library's
def _own(s):
    import moe_qw_repack_gb300.qw as Q
    kinds = {"bf16": Q.QW_T_BF16, "f16": Q.QW_T_F16, "f32": Q.QW_T_F32}
    X = s["X"]
    if s["op"] == "norm":
        K, R, got = s["K"], s["R"], {}
        fmt = Q.QW_A_MXFP8_G32 if s["q"] == "mxfp8" else Q.QW_A_INT8_TOKEN
        Q.qw_rmsnorm(kinds[s["x"]], X, X.stride(0), kinds.get(s["r"], Q.QW_T_BF16), R, K, s["R_out"],
                     K, s["W"], 0.0, EPS, s["rows"], K, s["Y"], K, fmt, s["codes"], s["scale"])
        if R is not None:
            got["h"] = s["R_out"]
        if s["y"]:
            got["y"] = s["Y"]
        if s["q"] == "mxfp8":
            got["codes"] = s["codes"].view(torch.float8_e4m3fn)
            got["scale"] = s["scale"].view(torch.float8_e8m0fnu)
        else:
            got["scale"] = s["scale"]
            got["values"] = torch.mul(s["codes"], s["scale"][:, None], out=s["values"])
        return got
    if s["op"] == "adapters":
        N = s["N"]
        Q.qgemm_lora(X, X.stride(0), s["A"], s["B"], s["scales"], s["ranks"], s["L"], s["R"],
                     s["ids"], s["base"], N, kinds[s["c"]], s["C"], N, s["M"], N, s["K"])
        return s["C"]
    layout = Q.QW_ROPE_HALF if s["layout"] == "half" else Q.QW_ROPE_INTERLEAVED
    n = s["heads"] * s["D"]
    Q.qw_rope(kinds[s["type"]], X, X.stride(0), s["Y"], n, s["T"], s["heads"], s["D"], s["rot"],
              layout, s["positions"], s["freqs"], s["attention"])
    return s["Y"]


def _plain(s):
    return {"norm": _plain_norm, "adapters": _plain_adapters, "rotary": _plain_rotary}[s["op"]](s)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- work, 64 bits
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}


def work(case):
    if case["op"] == "norm":
        n, K = case["rows"] * case["K"], case["K"]
        q = n + (n // 32 if case["q"] == "mxfp8" else 4 * case["rows"])
        return {"bytes": n * (_SIZE[case["x"]] + 2 * _SIZE[case["r"]] + 2 * case["y"]) + 2 * K + q,
                "flops": 6 * n}
    if case["op"] == "adapters":
        M, N, K, L, R = (case[k] for k in ("M", "N", "K", "L", "R"))
        some = min(L, M, 9) if case["runs"] else L * (1.0 - (1.0 - 1.0 / L) ** M)  # adapters met
        rank = R / 2 if case["mixed"] else R  # on average
        return {"bytes": 2 * M * K + 2 * some * rank * (K + N) + 2 * M * N * _SIZE[case["c"]],
                "flops": 2 * M * rank * (K + N)}
    T, n, part = case["T"], case["heads"] * case["D"], case["heads"] * case["rot"]
    return {"bytes": 2 * T * n * _SIZE[case["type"]] + 4 * T + 4 * case["rot"], "flops": 3 * T * part}


def _exact_norm(s):
    h, got = s["X"].double(), {}
    if s["R"] is not None:
        got["h"] = h + s["R"].double()
        h = got["h"].to(s["R"].dtype).double()  # (the sum is normalised as it is stored)
    y = s["W"].double() * h / (h.square().sum(dim=1, keepdim=True) / s["K"] + EPS).sqrt()
    if s["y"]:
        got["y"] = y
    if s["q"] == "mxfp8":
        g = y.unflatten(1, (-1, 32))
        power = torch.floor(torch.log2(g.abs().amax(dim=2))) - 8
        power = power.clamp(-127, 127)  # (a group of zeros: log2 gives -inf)
        v = (g * torch.exp2(-power)[:, :, None]).clamp(-448, 448)
        # E4M3: three bits behind the first, none below 2^-9
        ulp = torch.exp2((torch.floor(torch.log2(v.abs())).clamp(min=-6)) - 3)
        got["codes"] = (torch.round(v / ulp) * ulp).flatten(1)
        got["scale"] = torch.exp2(power)
    else:
        step = y.abs().amax(dim=1) / 127
        got["scale"] = step
        got["values"] = torch.round(y / step[:, None]) * step[:, None]
    return got


def _exact_adapters(s):
    out = s["base"].double()
    for a in range(s["L"]):
        r = int(s["ranks"][a])
        mine = torch.nonzero(s["ids"] == a)[:, 0]
        t = torch.einsum("mk,rk->mr", s["X"][mine].double(), s["A"][a, :r].double())
        out[mine] += s["scales"][a].double() * torch.einsum("mr,nr->mn", t, s["B"][a, :, :r].double())
    return out


def _exact_rotary(s):
    x = s["X"].double().reshape(s["T"], s["heads"], s["D"])
    n = s["rot"]
    pairs = x[:, :, :n].unflatten(2, (2, n // 2)).transpose(2, 3) if s["layout"] == "half" else \
        x[:, :, :n].unflatten(2, (n // 2, 2))
    angle = s["positions"].double()[:, None] * s["freqs"]
    turn = torch.polar(torch.full_like(angle, s["attention"]), angle)[:, None, :]
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    turned = turned.transpose(2, 3).flatten(2) if s["layout"] == "half" else turned.flatten(2)
    return torch.cat([turned, x[:, :, n:]], dim=2).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "adapters": _exact_adapters, "rotary": _exact_rotary}[s["op"]](s)
