"""Cases and plain forms of the operators on 4-bit weights.

A weight matrix [N, K] is held as 4-bit codes n, with a bf16 scale s and, in the
asymmetric form, a zero point z (0 .. 15; 8 in the symmetric form) for each row
and group of `group` columns.  A weight is the bf16 number round((n - z) * s).
Codes are uint8 [N, K/2]; the 32-bit word i of a row (8 codes) holds columns
8i, 8i+2, 8i+4, 8i+6 in its low four nibbles and 8i+1, 8i+3, 8i+5, 8i+7 in the
high ones.

  quantize   codes, scales and zero points of a bf16 matrix (and its values read
             back, the row lookup over every row)
  embed      rows of a table looked up by token id
  gemm       linear layer: column shards, row shards with their sum, SiluAndMul
  lm_head    logits of chosen hidden rows over the tied table, and greedy tokens

`own` false: elementary torch operations in fp32, rounded once at the end.
`own` true: the calls of this repository's library.
"""
import math

import torch

own = False


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one user's decode step: the merged QKV projection of a small model, where only latency counts
        dict(name="gemm one token qkv", op="gemm", M=1, N=4096, K=1024, group=128, zeros=False, tp=1, kind="column"),
        # decode of a few users: merged gate_up with SiluAndMul, two shards, asymmetric weights
        dict(name="gemm 8 tokens gate_up", op="gemm", M=8, N=12288, K=2048, group=64, zeros=True, tp=2, kind="silu"),
        # one token through the largest projection of a big model: the weights' bytes decide
        dict(name="gemm one token large", op="gemm", M=1, N=28672, K=8192, group=128, zeros=False, tp=1, kind="column"),
        # a decode batch through a down projection cut over its input columns, an odd batch
        dict(name="gemm 37 tokens down", op="gemm", M=37, N=4096, K=11264, group=128, zeros=True, tp=2, kind="row"),
        # a ragged chunk of a prompt, an output width that no tile divides, small groups
        dict(name="gemm 509 tokens odd", op="gemm", M=509, N=5003, K=5120, group=32, zeros=False, tp=1, kind="column"),
        # prefill of 8 prompts of 2048 tokens: gate_up with SiluAndMul
        dict(name="gemm 8 x 2k gate_up", op="gemm", M=16384, N=12288, K=2048, group=128, zeros=False, tp=1, kind="silu"),
        # the greedy step of a decode batch of 8 over this repository's vocabulary
        dict(name="lm_head 8 rows", op="lm_head", M=8, T=8, N=151936, K=1024, group=64, zeros=False, tp=1, last=False),
        # the last rows of a prefill's prompts, picked out of its hidden states, two shards
        dict(name="lm_head 65 of 4k", op="lm_head", M=65, T=4096, N=151936, K=1024, group=128, zeros=True, tp=2, last=True),
        # the embedding of one decode step
        dict(name="embed 64 ids", op="embed", M=64, N=151936, K=1024, group=64, zeros=False, tp=1),
        # the embedding of a prefill, two shards, asymmetric
        dict(name="embed 16k ids", op="embed", M=16384, N=151936, K=1024, group=32, zeros=True, tp=2),
        # loading: one projection of a layer
        dict(name="quantize 2k x 1k", op="quantize", N=2048, K=1024, group=128, zeros=False),
        # loading: the table of this repository's vocabulary
        dict(name="quantize table", op="quantize", N=151936, K=1024, group=32, zeros=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        group = rng.choice([32, 64, 128])
        tp = rng.choice([1, 1, 2, 4])
        c = dict(op=rng.choice(["gemm", "gemm", "gemm", "lm_head", "embed", "quantize"]), group=group,
                 zeros=rng.random() < 0.5)
        step = group * tp
        c["K"] = step * max(1, round(log(256, 12288) / step))
        if c["op"] == "quantize":
            c["N"] = log(100, 160000)
            if c["N"] * c["K"] > 151936 * 1024:
                continue
            return c
        c["tp"] = tp
        if c["op"] in ("embed", "lm_head"):
            c["N"] = 4 * log(250, 38000)
            c["M"] = log(1, 16384) if c["op"] == "embed" else log(1, 130)
            if c["N"] * c["K"] > 28672 * 8192 or c["M"] * c["K"] > 16384 * 1024:
                continue
            if c["op"] == "lm_head":
                c["last"] = rng.random() < 0.5
                c["T"] = c["M"] + (log(1, 2000) if c["last"] else 0)
            return c
        c["kind"] = rng.choice(["column", "row", "silu"])
        step = {"column": tp, "row": 1, "silu": 16 * tp}[c["kind"]]
        c["N"] = step * max(1, round(log(200, 30000) / step))
        c["M"] = log(1, 16384)
        if c["N"] * c["K"] > 28672 * 8192 or c["M"] * c["N"] * c["K"] > 16384 * 12288 * 2048:
            continue
        if c["M"] * (c["N"] + c["K"]) > 16384 * 16384:
            continue
        return c


def work(case):
    c = case
    N, K = c["N"], c["K"]
    weights = K / 2 + K // c["group"] * (2.5 if c["zeros"] else 2)      # bytes of one row; a zero point is 4 bits
    if c["op"] == "quantize":
        # in: the matrix; out: codes, scales, zeros; read back: those in, the values out
        return {"bytes": N * (2 * K + 2 * weights + 2 * K), "flops": 3 * N * K}
    if c["op"] == "embed":
        return {"bytes": c["M"] * (8 + weights + 2 * K), "flops": 2 * c["M"] * K}
    n_out = N // 2 if c.get("kind") == "silu" else N
    return {"bytes": N * weights + 2 * c["M"] * (K + n_out), "flops": 2 * c["M"] * N * K}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

_PLACE = (0, 4, 1, 5, 2, 6, 3, 7)         # nibble of column 8i + j


def _put(n):
    """Codes (0 .. 15) [.., K] as bytes [.., K/2]."""
    n = n.view(*n.shape[:-1], -1, 8).int()
    word = torch.zeros_like(n[..., 0])
    for j, p in enumerate(_PLACE):
        word |= n[..., j] << (4 * p)
    return word.view(torch.uint8)


def _take(codes):
    """Bytes [.., K/2] as codes (0 .. 15) [.., K]."""
    word = codes.view(torch.int32)
    return torch.stack([(word >> (4 * p)) & 15 for p in _PLACE], -1).view(*codes.shape[:-1], -1)


def _quantize(w, group, zeros):
    """(codes 0 .. 15 [N, K], scales bf16, zeros uint8 or None) of a bf16 matrix."""
    x = w.float().view(w.shape[0], -1, group)
    if zeros:
        lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15.0).bfloat16()
        d = s.float().masked_fill(s == 0, 1.0)
        z = torch.round(-lo / d).clamp(0, 15)
        n = (torch.round(x / d[..., None]) + z[..., None]).clamp(0, 15)
        return n.view(w.shape), s, z.to(torch.uint8)
    s = (x.abs().amax(-1) / 7.0).bfloat16()
    d = s.float().masked_fill(s == 0, 1.0)
    n = torch.round(x / d[..., None]).clamp(-8, 7) + 8.0
    return n.view(w.shape), s, None


def _values(n, scales, zeros, group):
    """The weights as bf16 numbers, in fp32."""
    n = n.float().view(*n.shape[:-1], -1, group)
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((n - z) * scales.float()[..., None]).bfloat16().float().view(*n.shape[:-2], -1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    N, K = c["N"], c["K"]
    # weights of a trained matrix: near normal, rows of different size, a few large input columns
    rows = torch.exp(0.3 * normal(N, 1))
    cols = torch.exp(0.3 * normal(1, K))
    w = (0.02 * rows * cols * normal(N, K)).bfloat16()
    s = {"case": dict(c)}
    if c["op"] == "quantize":
        s["w"] = w
        s["codes"] = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(N, K // c["group"], dtype=torch.bfloat16, device="cuda")
        s["zeros"] = torch.empty(N, K // c["group"], dtype=torch.uint8, device="cuda") if c["zeros"] else None
        s["ids"] = torch.arange(N, device="cuda")
        s["out"] = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
        return s
    if c.get("kind") == "row":
        # shard r: the input columns r * K/tp .. (r+1) * K/tp - 1
        w = w.view(N, c["tp"], K // c["tp"]).transpose(0, 1).reshape(c["tp"] * N, K // c["tp"])
    n, s["scales"], s["zeros"] = _quantize(w, c["group"], c["zeros"])
    del w
    s["codes"] = _put(n)
    if c["op"] == "embed":
        s["ids"] = torch.randint(0, N, (c["M"],), generator=g, device="cuda")
        s["out"] = torch.empty(c["M"], K, dtype=torch.bfloat16, device="cuda")
        return s
    # activations behind a norm: near normal, a few columns much larger
    big = 1.0 + 15.0 * (torch.rand(1, K, generator=g, device="cuda") < 0.004).float()
    x = normal(c["T"] if c["op"] == "lm_head" else c["M"], K) * big
    if c["op"] == "lm_head":
        s["last"] = None
        if c["last"]:
            s["last"] = torch.randperm(c["T"], generator=g, device="cuda")[:c["M"]].sort().values.int()
        # hidden states that point at one token, as those of a model that is sure of its next word
        at = s["last"].long() if c["last"] else torch.arange(c["M"], device="cuda")
        tok = torch.randint(0, N, (c["M"],), generator=g, device="cuda")
        v = _values(n[tok], s["scales"][tok], None if s["zeros"] is None else s["zeros"][tok], c["group"])
        x[at] = 0.3 * x[at] + 2.0 * v / v.square().mean(-1, keepdim=True).sqrt()
        s["logits"] = torch.empty(c["M"], N, dtype=torch.bfloat16, device="cuda")
        s["tokens"] = torch.empty(c["M"], dtype=torch.int64, device="cuda")
    else:
        s["out"] = torch.empty(c["M"], N // 2 if c["kind"] == "silu" else N, dtype=torch.bfloat16, device="cuda")
    s["x"] = x.bfloat16()
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _weights(s):
    return _values(_take(s["codes"]), s["scales"], s["zeros"], s["case"]["group"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        n, scales, zeros = _quantize(s["w"], c["group"], c["zeros"])
        out = {"values": _values(n, scales, zeros, c["group"]).bfloat16(), "scales": scales}
        return {**out, "zeros": zeros} if c["zeros"] else out
    if c["op"] == "embed":
        zeros = None if s["zeros"] is None else s["zeros"][s["ids"]]
        return {"out": _values(_take(s["codes"][s["ids"]]), s["scales"][s["ids"]], zeros, c["group"]).bfloat16()}
    if c["op"] == "lm_head":
        x = s["x"][:c["M"]] if s["last"] is None else s["x"][s["last"].long()]
        y = (x.float() @ _weights(s).T).bfloat16()
        return {"logits": y, "tokens": y.argmax(-1)}
    x, w = s["x"].float(), _weights(s)
    tp = c["tp"]
    if c["kind"] == "row":
        y = sum(xr @ wr.T for xr, wr in zip(x.chunk(tp, 1), w.chunk(tp, 0)))
        return {"out": y.bfloat16()}
    y = x @ w.T
    if c["kind"] == "silu":
        gate, up = y.view(c["M"], tp, 2, -1).unbind(2)      # shard r's columns: gate_r, up_r
        y = (gate / (1.0 + torch.exp(-gate)) * up).reshape(c["M"], -1)
    return {"out": y.bfloat16()}


# ----------------------------------------------------------------------------
# this repository's operators
# ----------------------------------------------------------------------------

def _run_own(s):
    from qwen3_transformer_forward_gb300 import lib as L
    c = s["case"]
    if c["op"] == "quantize":
        L.w4_quantize(s["w"], c["group"], s["codes"], s["scales"], s["zeros"])
        L.w4_embed_vocab(s["ids"], s["codes"], s["scales"], s["zeros"], c["group"], 1, s["out"])
        out = {"values": s["out"], "scales": s["scales"]}
        return {**out, "zeros": s["zeros"]} if c["zeros"] else out
    if c["op"] == "embed":
        L.w4_embed_vocab(s["ids"], s["codes"], s["scales"], s["zeros"], c["group"], c["tp"], s["out"])
        return {"out": s["out"]}
    if c["op"] == "lm_head":
        if "workspace" not in s:
            size = L.w4_lm_head_workspace_size(c["M"], c["N"], c["K"], c["tp"])
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        L.w4_lm_head(s["x"], s["last"], c["M"], s["codes"], s["scales"], s["zeros"], c["group"], c["tp"], s["logits"],
                     s["tokens"], s["workspace"])
        return {"logits": s["logits"], "tokens": s["tokens"]}
    mode = L.QW_GEMM_ROW_REDUCE if c["kind"] == "row" else L.QW_GEMM_COLUMN
    epilogue = L.QW_EPI_SILU_MUL if c["kind"] == "silu" else L.QW_EPI_NONE
    if "workspace" not in s:
        size = L.w4_gemm_workspace_size(c["M"], c["N"], c["K"], c["tp"], mode, epilogue)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    L.w4_gemm(s["x"], s["codes"], s["scales"], s["zeros"], s["out"], c["N"], c["group"], c["tp"], mode, epilogue,
              s["workspace"])
    return {"out": s["out"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# from the definition, in 64 bits
# ----------------------------------------------------------------------------

def _columns(codes):
    """Codes column by column, from the bytes: byte b of a word holds two nibbles of its columns."""
    rows, half = codes.shape
    b = codes.view(rows, half // 4, 4)
    out = torch.empty(rows, half // 4, 8, dtype=torch.float64, device=codes.device)
    for j in range(8):
        nib = (j & 1) * 4 + j // 2
        byte = b[:, :, nib // 2]
        out[:, :, j] = (byte >> 4 if nib & 1 else byte & 15).double()
    return out.reshape(rows, half * 2)


def _matrix(s):
    c = s["case"]
    n = _columns(s["codes"])
    z = torch.full_like(s["scales"], 8.0).double() if s["zeros"] is None else s["zeros"].double()
    n -= z.repeat_interleave(c["group"], 1)
    n *= s["scales"].double().repeat_interleave(c["group"], 1)
    return n.bfloat16().double()      # (n - z) * s has 12 bits: fp32 on the way holds it whole


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantize":
        w = s["w"].double().view(c["N"], -1, c["group"])
        if c["zeros"]:
            lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
            scale = ((hi - lo) / 15).bfloat16().double()
        else:
            scale = (w.abs().amax(-1) / 7).bfloat16().double()
        d = torch.where(scale == 0, torch.ones_like(scale), scale)[..., None]
        q = torch.round(w / d)
        if c["zeros"]:
            zero = torch.clamp(torch.round(-lo[..., None] / d), 0, 15)
            q = torch.clamp(q + zero, 0, 15) - zero
        else:
            q = torch.clamp(q, -8, 7)
        out = {"values": (q * scale[..., None]).bfloat16().double().view(c["N"], -1), "scales": scale}
        return {**out, "zeros": zero[..., 0].to(torch.uint8)} if c["zeros"] else out
    if c["op"] == "embed":
        return {"out": _matrix(s)[s["ids"]]}
    x = s["x"].double()
    if c["op"] == "lm_head":
        x = x[:c["M"]] if s["last"] is None else x[s["last"].long()]
        y = x @ _matrix(s).T
        return {"logits": y, "tokens": y.argmax(-1)}
    w = _matrix(s)
    if c["kind"] == "row":
        w = w.view(c["tp"], c["N"], -1).permute(1, 0, 2).reshape(c["N"], c["K"])
    y = x @ w.T
    if c["kind"] == "silu":
        il = c["N"] // 2 // c["tp"]
        pick = torch.arange(c["N"] // 2, device="cuda")
        gate = y[:, pick // il * 2 * il + pick % il]
        up = y[:, pick // il * 2 * il + il + pick % il]
        y = gate * torch.sigmoid(gate) * up
    return {"out": y}
