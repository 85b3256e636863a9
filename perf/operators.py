"""Cases of the INT8 serving operators: the INT8 product, the gated INT8 projections and the
log probabilities, each in its plain form (elementary torch operations in 32 bits) and, where
``own`` is true, through the library's entry points.

  product   C = a_scale * w_scale * (A_q W^T) + bias, from BF16 activations (quantised per token
            within the call) or from INT8 activations with their scales
  gated     Y = silu(gate projection) * (up projection) on the same integers
  logprobs  log probability and rank of a given token, entropy and top alternatives of each row
"""
import math

import torch

own = False

FLT_MAX = 3.4028234663852886e38


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through a 4096 -> 14336 projection (decode: latency and the weight stream)
        dict(name="product token", op="product", M=1, N=14336, K=4096, a="bf16", out="bf16",
             bias=False, pad=0),
        # a decode batch through the down projection (few output rows, long K)
        dict(name="product batch 16", op="product", M=16, N=4096, K=14336, a="bf16", out="bf16",
             bias=False, pad=0),
        # an LM head of odd width over a batch, FP32 logits out, activations already quantised
        dict(name="product head 64", op="product", M=64, N=32003, K=4096, a="int8", out="f32",
             bias=False, pad=0),
        # a ragged prompt with a bias, rows taken out of a wider tensor
        dict(name="product ragged 333", op="product", M=333, N=1000, K=1040, a="bf16", out="bf16",
             bias=True, pad=48),
        # a long prompt
        dict(name="product prompt 4096", op="product", M=4096, N=14336, K=4096, a="bf16",
             out="bf16", bias=False, pad=0),
        # one token through the gate and up projections of a 4096 / 14336 block
        dict(name="gated token", op="gated", M=1, I=14336, K=4096, a="bf16", bias=False, pad=0),
        # a speculative or mixed batch on a small block of odd width
        dict(name="gated ragged 77", op="gated", M=77, I=1111, K=1040, a="int8", bias=True, pad=32),
        # a long prompt through the gate and up projections
        dict(name="gated prompt 4096", op="gated", M=4096, I=14336, K=4096, a="bf16", bias=False,
             pad=0),
        # the sampled token of one sequence, five alternatives
        dict(name="logprobs token", op="logprobs", T=1, V=131072, dtype="bf16", topk=5,
             masked=0.0, pad=0),
        # a decode batch under a grammar mask, FP32 logits of odd width (one row fully masked)
        dict(name="logprobs batch 64", op="logprobs", T=64, V=32003, dtype="f32", topk=20,
             masked=0.9, pad=0),
        # scoring a prompt of odd vocabulary out of a padded logits tensor
        dict(name="logprobs ragged 777", op="logprobs", T=777, V=50021, dtype="f16", topk=8,
             masked=0.0, pad=43),
        # scoring a long prompt
        dict(name="logprobs prompt 4096", op="logprobs", T=4096, V=131072, dtype="bf16", topk=20,
             masked=0.0, pad=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "gated", "logprobs"])
    if op == "logprobs":
        V = _log_int(rng, 300, 262144)
        T = _log_int(rng, 1, max(1, min(8192, 4096 * 131072 // V)))
        return dict(op=op, T=T, V=V, dtype=rng.choice(["bf16", "f16", "f32"]),
                    topk=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.0, 0.5, 0.95]),
                    pad=rng.choice([0, 0, 1, 13, 64]))
    K = 16 * _log_int(rng, 4, 1024)
    M = _log_int(rng, 1, 8192)
    a, bias, pad = rng.choice(["bf16", "int8"]), rng.random() < 0.5, 16 * rng.choice([0, 0, 1, 5])
    if op == "gated":
        cap = 4096 * 14336 * 4096 // (M * K)
        return dict(op=op, M=M, I=_log_int(rng, 16, max(17, min(16384, cap))), K=K, a=a, bias=bias,
                    pad=pad)
    cap = 4096 * 14336 * 4096 // (M * K)
    return dict(op=op, M=M, N=_log_int(rng, 16, max(17, min(40000, cap))), K=K, a=a,
                out=rng.choice(["bf16", "bf16", "f32"]), bias=bias, pad=pad)


# ----------------------------------------------------------------------------- the inputs
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _codes(shape, gen):
    """INT8 codes as quantised weights and activations have them: a rounded normal."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.mul_(32.0).round_().clamp_(-127.0, 127.0).to(torch.int8)


def _activations(M, K, pad, a, gen):
    """BF16 rows of different magnitude with a few loud channels, or INT8 codes and scales;
    rows of a wider tensor where pad > 0."""
    if a == "int8":
        wide = _codes((M, K + pad), gen)
        scale = torch.rand(M, generator=gen, device="cuda") * 0.04 + 0.01
        return wide[:, :K], scale
    wide = torch.randn((M, K + pad), generator=gen, device="cuda")
    wide *= torch.exp2(torch.randint(-3, 4, (M, 1), generator=gen, device="cuda").float())
    loud = torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")
    wide[:, loud] *= 8.0
    return wide.to(torch.bfloat16)[:, :K], None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "logprobs":
        T, V, pad = case["T"], case["V"], case["pad"]
        wide = torch.empty((T, V + pad), dtype=_DTYPES[case["dtype"]], device="cuda")
        for i in range(0, T, 512):  # in parts: the FP32 draw is up to four times the logits
            part = torch.randn((min(512, T - i), V + pad), generator=gen, device="cuda")
            wide[i:i + 512] = part.mul_(2.5)
        logits = wide[:, :V]
        peaks = torch.randint(0, V, (T, 8), generator=gen, device="cuda")
        rise = torch.rand((T, 8), generator=gen, device="cuda") * 6.0 + 6.0
        logits.scatter_(1, peaks, rise.to(logits.dtype))
        tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
        likely = torch.rand(T, generator=gen, device="cuda") < 0.75
        tokens = torch.where(likely, peaks[:, 0], tokens)
        if case["masked"] > 0:
            gone = torch.rand((T, V), generator=gen, device="cuda") < case["masked"]
            logits.masked_fill_(gone, float("-inf"))
            if T > 2:
                logits[T // 2] = float("-inf")  # a mask that leaves nothing
        k = case["topk"]
        s.update(logits=logits, tokens=tokens.to(torch.int32),
                 lp=torch.empty(T, device="cuda"),
                 rank=torch.empty(T, dtype=torch.int32, device="cuda"),
                 ent=torch.empty(T, device="cuda"),
                 top=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                 top_lp=torch.empty((T, k), device="cuda"))
        return s
    M, K = case["M"], case["K"]
    N = 2 * case["I"] if case["op"] == "gated" else case["N"]
    A, a_scale = _activations(M, K, case["pad"], case["a"], gen)
    W = _codes((N, K), gen)
    w_scale = (torch.rand(N, generator=gen, device="cuda") + 0.5) / (32.0 * math.sqrt(K))
    bias = None
    if case["bias"]:
        bias = torch.randn(N, generator=gen, device="cuda").to(torch.bfloat16)
    out = _DTYPES[case["out"]] if case["op"] == "product" else torch.bfloat16
    cols = N if case["op"] == "product" else case["I"]
    s.update(A=A, a_scale=a_scale, W=W, w_scale=w_scale, bias=bias,
             C=torch.empty((M, cols), dtype=out, device="cuda"))
    return s


# ----------------------------------------------------------------------------- plain forms
def _plain_sums(s):
    """The scaled integer product in FP32, before the output's rounding."""
    if s["a_scale"] is None:
        x = s["A"].float()
        amax = x.abs().amax(dim=1, keepdim=True)
        q = torch.round(x * (127.0 / amax).clamp(max=FLT_MAX))
        sa = amax / 127.0
    else:
        q = s["A"].float()
        sa = s["a_scale"][:, None]
    c = (q @ s["W"].float().t()) * (sa * s["w_scale"][None, :])
    return c if s["bias"] is None else c + s["bias"].float()


def _plain_logprobs(s):
    x = s["logits"].float()
    V, k = s["V"], s["topk"]
    m = x.amax(dim=1, keepdim=True)
    some = m > float("-inf")  # rows whose mask leaves something
    d = torch.where(some, x - torch.where(some, m, torch.zeros_like(m)), torch.full_like(m, float("-inf")))
    e = torch.exp(d)
    z = e.sum(dim=1, keepdim=True)
    log_z = torch.log(z)
    ent = log_z[:, 0] - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(dim=1) / z[:, 0]
    ent = torch.where(some[:, 0], ent, torch.zeros_like(ent))
    none = torch.full_like(x[:, :1], float("-inf"))
    tok = s["tokens"].long()[:, None]
    xt = x.gather(1, tok)
    lp = torch.where(some, d.gather(1, tok) - log_z, none)[:, 0]
    ids = torch.arange(V, device=x.device)
    rank = 1 + (x > xt).sum(dim=1) + ((x == xt) & (ids < tok)).sum(dim=1)
    # order by value, equal values by the lower id: the value's bits as an ordered integer above
    # the complement of the id (-0 and 0 are equal: adding 0 makes them the same)
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits) * (1 << 32) + (V - 1 - ids)
    top = V - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)
    top_lp = torch.where(some, d.gather(1, top) - log_z, none)
    return dict(lp=lp, rank=rank.int(), ent=ent, top=top.int(), top_lp=top_lp)


def _plain(s):
    if s["op"] == "logprobs":
        return _plain_logprobs(s)
    c = _plain_sums(s)
    if s["op"] == "gated":
        g, u = c[:, :s["I"]], c[:, s["I"]:]
        c = g / (1.0 + torch.exp(-g)) * u
    return c.to(s["C"].dtype)


# ----------------------------------------------------------------------------- the library's
def _own(s):
    import moe_qw_repack_gb300.qw as Q
    if s["op"] == "logprobs":
        kind = {"bf16": Q.QW_T_BF16, "f16": Q.QW_T_F16, "f32": Q.QW_T_F32}[s["dtype"]]
        Q.qw_logprobs(kind, s["logits"], s["logits"].stride(0), s["T"], s["V"], s["tokens"],
                      s["topk"], s["lp"], s["rank"], s["ent"], s["top"], s["top_lp"])
        return dict(lp=s["lp"], rank=s["rank"], ent=s["ent"], top=s["top"], top_lp=s["top_lp"])
    afmt = Q.QW_A_BF16 if s["a_scale"] is None else Q.QW_A_INT8_TOKEN
    M, K, C = s["M"], s["K"], s["C"]
    N = 2 * s["I"] if s["op"] == "gated" else s["N"]
    if "workspace" not in s:  # kept with the plan, as a server keeps it
        n = Q.qgemm_int8_workspace_size(afmt, M, N, K)
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    ws = s["workspace"]
    if s["op"] == "gated":
        Q.qgemm_int8_gated(afmt, s["A"], s["A"].stride(0), s["a_scale"], s["W"], s["w_scale"],
                           s["bias"], C, s["I"], M, s["I"], K, ws, ws.numel())
    else:
        kind = Q.QW_T_F32 if s["out"] == "f32" else Q.QW_T_BF16
        Q.qgemm_int8(afmt, s["A"], s["A"].stride(0), s["a_scale"], s["W"], s["w_scale"], s["bias"],
                     kind, C, s["N"], M, s["N"], K, ws, ws.numel())
    return C


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- work, 64 bits
def work(case):
    if case["op"] == "logprobs":
        T, V = case["T"], case["V"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * V * size + T * (16 + 8 * case["topk"]), "flops": 4 * T * V}
    M, K = case["M"], case["K"]
    gated = case["op"] == "gated"
    N = 2 * case["I"] if gated else case["N"]
    a = M * K * 2 if case["a"] == "bf16" else M * K + 4 * M
    c = 2 * M * case["I"] if gated else M * N * (4 if case["out"] == "f32" else 2)
    return {"bytes": a + N * K + 4 * N + (2 * N if case["bias"] else 0) + c, "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        lp, ent, top_lp = [], [], []
        for i in range(0, case["T"], 256):
            x = s["logits"][i:i + 256].double()
            lse = torch.logsumexp(x, dim=1, keepdim=True)
            logp = torch.where(torch.isfinite(lse), x - lse, torch.full_like(x, float("-inf")))
            p = logp.exp()
            lp.append(logp.gather(1, s["tokens"][i:i + 256].long()[:, None])[:, 0])
            ent.append(torch.special.entr(p).sum(dim=1))
            top_lp.append(logp.topk(case["topk"], dim=1).values)
        return dict(lp=torch.cat(lp), rank=None, ent=torch.cat(ent), top=None,
                    top_lp=torch.cat(top_lp))
    A = s["A"].double()
    if s["a_scale"] is None:
        step = A.abs().amax(dim=1) / 127.0
        A = torch.where(step[:, None] > 0, torch.round(A / step[:, None]), torch.zeros_like(A))
    else:
        step = s["a_scale"].double()
    C = torch.einsum("mk,nk->mn", A, s["W"].double())
    C = C * step[:, None] * s["w_scale"].double()
    if s["bias"] is not None:
        C += s["bias"].double()
    if case["op"] == "gated":
        g, u = C.split(case["I"], dim=1)
        C = g * torch.sigmoid(g) * u
    return C
