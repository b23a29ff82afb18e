"""Measured cases of the MXFP4 operators and of the router's balance loss.

MXFP4 (OCP Microscaling Formats v1.0) holds E2M1 values in blocks of 32 under
one E8M0 (power of two) scale.  For a block with largest magnitude a the scale
is 2^(floor(log2 a) - 2), no less than 2^-127, and each element is x / scale
rounded to the E2M1 grid {0, .5, 1, 1.5, 2, 3, 4, 6} (nearest, ties to even,
clamped at 6).  The last block of a row whose length is no multiple of 32 is
filled up with zeros.

The operators, by a case's "op":

* quantize: a matrix to MXFP4 and read back.
* transpose: the same with the blocks along the columns (the matrix's
  transpose, which a product over the rows takes), read back.
* linear: y = q(x) W^T with x quantised in the call and MXFP4 weights.
* experts: the same per expert over permuted rows: y[r] = weight[r] *
  q(x[perm[r]]) W_e^T for the rows r of expert e's segment.
* weight_grad: dW = q(dy^T) q(x^T)^T, both quantised along the tokens.
* balance: the router's load-balance loss, per-expert counts and the gradient
  of the loss with respect to the logits.

Weights come as a user's program keeps them: packed codes, two a byte with
the even element in the low nibble, and scales in the tiled layout (512-byte
atoms of 128 rows x 4 blocks, row r and block b at (r % 32) * 16 + (r / 32) *
4 + b, atoms row tile by row tile).
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the activations of one decoding step of the 6144-wide layer
        dict(name="quantize 16 x 6144 bf16", op="quantize", rows=16, cols=6144, dtype="bf16"),
        # a prompt's activations in half precision, rows that end inside a block
        dict(name="quantize 8191 x 6100 fp16", op="quantize", rows=8191, cols=6100, dtype="fp16"),
        # offline: gate and up of 16 experts in one call
        dict(name="quantize 65536 x 6144 bf16", op="quantize", rows=65536, cols=6144, dtype="bf16"),
        # a training step's activations, blocks along the tokens
        dict(name="transpose 8192 x 6144 bf16", op="transpose", rows=8192, cols=6144, dtype="bf16"),
        # a ragged micro-batch of fp32 gradients
        dict(name="transpose 1001 x 2049 fp32", op="transpose", rows=1001, cols=2049, dtype="fp32"),
        # one token through a hidden-to-hidden projection
        dict(name="linear 1 x 6144 x 6144 bf16", op="linear", M=1, N=6144, K=6144, dtype="bf16"),
        # a small batch, odd sizes throughout
        dict(name="linear 37 x 5001 x 2010 fp16", op="linear", M=37, N=5001, K=2010, dtype="fp16"),
        # a prompt through gate and up
        dict(name="linear 8192 x 4096 x 6144 bf16", op="linear", M=8192, N=4096, K=6144, dtype="bf16"),
        # 64 tokens, top-8 of 16 experts, the down projection with its routing weights
        dict(name="experts 64 x 6144 x 2048 bf16", op="experts", T=64, k=8, E=16, N=6144, K=2048, dtype="bf16"),
        # the weight gradient of a training step
        dict(name="weight_grad 4096: 2048 x 6144", op="weight_grad", T=4096, N=2048, K=6144, dtype="bf16"),
        # routing statistics of one decoding step
        dict(name="balance 16 x 80 sigmoid", op="balance", T=16, E=80, k=8, S=1, masked=False, score="sigmoid",
             dtype="fp32"),
        # a training batch of packed sequences with padding
        dict(name="balance 65531 x 128 softmax", op="balance", T=65531, E=128, k=8, S=17, masked=True,
             score="softmax", dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "transpose", "linear", "linear", "experts", "weight_grad", "balance", "balance"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("quantize", "transpose"):
        cols = _log_int(rng, 33, 16384)
        rows = _log_int(rng, 1, min(65536, 200000000 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype)
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 4096), K=_log_int(rng, 64, 6144),
                    dtype=rng.choice(["bf16", "fp16"]))
    if op == "experts":
        E = rng.choice([4, 8, 16, 32])
        return dict(op=op, T=_log_int(rng, 1, 1024), k=rng.randint(1, 4), E=E, N=128 * _log_int(rng, 1, 24),
                    K=_log_int(rng, 64, 2048), dtype=rng.choice(["bf16", "fp16"]))
    if op == "weight_grad":
        return dict(op=op, T=_log_int(rng, 16, 8192), N=_log_int(rng, 64, 2500), K=_log_int(rng, 64, 6144),
                    dtype=rng.choice(["bf16", "fp16"]))
    E = _log_int(rng, 8, 512)
    T = _log_int(rng, 1, 65536 if E <= 128 else 16384)
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=rng.choice([1, 1, min(T, 5), min(T, 64)]),
                masked=rng.choice([True, False]), score=rng.choice(["sigmoid", "softmax"]),
                dtype=rng.choice(["fp32", "fp32", "bf16"]))


def _padded(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _mx_bytes(rows, cols):
    """Codes and scales of a matrix, without the tiled layout's padding rows."""
    return rows * _padded(cols) * (0.5 + 1 / BLOCK)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op in ("quantize", "transpose"):
        r, c = case["rows"], case["cols"]
        q = _mx_bytes(r, c) if op == "quantize" else _mx_bytes(c, r)
        return {"bytes": 2 * r * c * size + 2 * q, "flops": 0}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size + _mx_bytes(N, K) + M * N * size, "flops": 2 * M * N * K}
    if op == "experts":
        P, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
        # the experts that T * k uniform choices without repetition per token are expected to reach
        hit = E * (1 - (1 - case["k"] / E) ** case["T"])
        return {"bytes": case["T"] * K * size + hit * _mx_bytes(N, K) + P * (N * size + 8), "flops": 2 * P * N * K}
    if op == "weight_grad":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * (N + K) * size + N * K * 4, "flops": 2 * T * N * K}
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    # logits and choices in, gradient and the per-sequence counts out
    return {"bytes": T * (2 * E * size + 4 * k + (1 if case["masked"] else 0)) + 4 * S * E, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, dtype, std=1.0, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda") * std
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < outliers, 20 * x, x)
    return x.to(dtype)


def _pack(values_code):
    """[rows, cols] 4-bit codes -> two a byte, the even element in the low nibble."""
    c = values_code.to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _tile_index(rows, blocks, device):
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(blocks, device=device)[None, :]
    atoms = (blocks + 3) // 4
    return ((r // 128) * atoms + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4


def _tile(scales):
    """[rows, blocks] scale bytes -> the tiled layout (zero in its padding)."""
    rows, blocks = scales.shape
    out = torch.zeros((rows + 127) // 128 * ((blocks + 3) // 4) * 512, dtype=torch.uint8, device=scales.device)
    out[_tile_index(rows, blocks, scales.device).reshape(-1)] = scales.reshape(-1)
    return out


def _weights(gen, rows, K):
    """MXFP4 weights of N(0, 0.02): (codes, tiled scales)."""
    w = _normal(gen, (rows, K), torch.bfloat16, std=0.02)
    code, exponent = _encode(w)
    return _pack(code), _tile((exponent + 127).to(torch.uint8))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dtype = case["op"], DTYPES[case["dtype"]]
    st = dict(case, dtype=dtype)
    if op in ("quantize", "transpose"):
        st["x"] = _normal(gen, (case["rows"], case["cols"]), dtype, outliers=0.001)
    elif op == "linear":
        st["x"] = _normal(gen, (case["M"], case["K"]), dtype, outliers=0.001)
        st["codes"], st["scales"] = _weights(gen, case["N"], case["K"])
    elif op == "experts":
        T, k, E = case["T"], case["k"], case["E"]
        st["x"] = _normal(gen, (T, case["K"]), dtype, outliers=0.001)
        st["codes"], st["scales"] = _weights(gen, E * case["N"], case["K"])
        # a router's choice: pairs in expert, then token order, segments padded to 128 rows
        expert = torch.rand((T, E), generator=gen, device="cuda").topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(expert, stable=True).indices
        counts = torch.bincount(expert, minlength=E)
        padded = (counts + 127) // 128 * 128
        offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
        first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])[:E]
        sorted_expert = expert[order]
        rows = offsets[sorted_expert] + torch.arange(T * k, device="cuda") - first[sorted_expert]
        cap = (T * k + 127 * E + 127) // 128 * 128
        st["perm"] = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
        st["perm"][rows] = (order // k).to(torch.int32)
        st["row_weight"] = torch.zeros(cap, device="cuda")
        st["row_weight"][rows] = torch.rand(T * k, generator=gen, device="cuda")
        st["offsets"], st["counts"] = offsets.to(torch.int32), counts.to(torch.int32)
        st["rows"], st["most"] = rows, int(counts.max())
        st["y"] = torch.zeros((cap, case["N"]), dtype=dtype, device="cuda")
    elif op == "weight_grad":
        st["x"] = _normal(gen, (case["T"], case["K"]), dtype, outliers=0.001)
        st["dy"] = _normal(gen, (case["T"], case["N"]), dtype, std=1e-2)
    else:
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        logits = _normal(gen, (T, E), dtype, std=1.5) + _normal(gen, (E,), dtype, std=0.5)
        st["logits"] = logits
        st["topk_idx"] = logits.float().topk(k, dim=1).indices.to(torch.int32)
        cuts = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda").sort().values
        st["seq_offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        st["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.9 if case["masked"] else None
        st["coeff"] = 1e-2
        st["grad_loss"] = torch.rand(1, generator=gen, device="cuda") + 0.5
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _encode(x):
    """(4-bit codes [rows, padded], scale exponents [rows, blocks]) of a matrix."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _padded(cols) - cols)).reshape(rows, -1, BLOCK)
    amax = x.abs().amax(dim=2)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
    y = torch.ldexp(x, -exponent[:, :, None])
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(x)
    return code.reshape(rows, -1), exponent


def _values(code, exponent):
    """fp32 values of codes [rows, padded] under exponents [rows, blocks]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    grid = torch.cat([grid, -grid])
    v = grid[code.long()].reshape(code.shape[0], -1, BLOCK)
    return torch.ldexp(v, exponent[:, :, None]).reshape(code.shape[0], -1)


def _quantized(x):
    return _values(*_encode(x))


def _weight_values(codes, scales):
    """fp32 values [rows, padded] of packed codes with tiled scales."""
    rows, half = codes.shape
    code = torch.stack([codes & 15, codes >> 4], dim=2).reshape(rows, 2 * half)
    blocks = 2 * half // BLOCK
    exponent = scales[_tile_index(rows, blocks, codes.device)].to(torch.int32) - 127
    return _values(code, exponent)


def _plain_balance(st):
    logits = st["logits"].float()
    T, E = logits.shape
    k, S = st["k"], st["S"]
    keep = torch.ones(T, dtype=torch.bool, device=logits.device) if st["mask"] is None else st["mask"]
    seq = torch.bucketize(torch.arange(T, device=logits.device), st["seq_offsets"][1:].long(), right=True)
    sig = torch.sigmoid(logits)
    p = torch.softmax(logits, dim=1) if st["score"] == "softmax" else sig / sig.sum(dim=1, keepdim=True)
    p = p * keep[:, None]
    chosen = torch.zeros((T, E), device=logits.device).scatter_add_(
        1, st["topk_idx"].long(), keep[:, None].expand(T, k).float())
    tokens = torch.zeros(S, dtype=torch.float64, device=logits.device).index_add_(0, seq, keep.double())
    # sums over up to T tokens: taken in 64 bits, rounded once
    counts = torch.zeros((S, E), dtype=torch.float64, device=logits.device).index_add_(0, seq, chosen.double())
    mean = torch.zeros((S, E), dtype=torch.float64, device=logits.device).index_add_(0, seq, p.double())
    mean = mean / tokens.clamp(min=1)[:, None]
    share = counts * E / (k * tokens.clamp(min=1)[:, None])
    scale = st["coeff"] / (tokens > 0).sum().clamp(min=1)
    loss = scale * (share * mean).sum()
    f = share.float()[seq]
    g = (st["grad_loss"] * (scale / tokens.clamp(min=1)).float()[seq])[:, None]
    d = g * p * (f - (p * f).sum(dim=1, keepdim=True))
    if st["score"] == "sigmoid":
        d = d * (1 - sig)
    return dict(loss=loss.float().reshape(1), counts=counts.to(torch.int32), probs=mean.float(),
                dlogits=d.to(st["logits"].dtype))


def _plain(st):
    op = st["op"]
    if op == "quantize":
        return _quantized(st["x"])[:, :st["cols"]].to(st["dtype"])
    if op == "transpose":
        return _quantized(st["x"].t())[:, :st["rows"]].to(st["dtype"])
    if op == "linear":
        return (_quantized(st["x"]) @ _weight_values(st["codes"], st["scales"]).t()).to(st["dtype"])
    if op == "experts":
        E, N = st["E"], st["N"]
        x = _quantized(st["x"])
        w = _weight_values(st["codes"], st["scales"]).reshape(E, N, -1)
        # every expert's rows side by side, as many as the fullest expert has
        row = (st["offsets"][:E, None] + torch.arange(st["most"], device=x.device)).clamp(max=st["perm"].numel() - 1)
        y = torch.bmm(x[st["perm"][row].clamp(min=0).long()], w.transpose(1, 2))
        y = y * st["row_weight"][row][:, :, None]
        real = torch.arange(st["most"], device=x.device) < st["counts"][:, None]
        st["y"][row[real].long()] = y[real].to(st["dtype"])
        return st["y"]
    if op == "weight_grad":
        return _quantized(st["dy"].t()) @ _quantized(st["x"].t()).t()
    return _plain_balance(st)


def run(state):
    st = state
    if not own:
        return _plain(st)
    from nvfp4_w4a4_quantized_moe_b200 import capi

    op = st["op"]
    if op == "quantize":
        return capi.mxfp4_dequantize(capi.mxfp4_quantize(st["x"]), dtype=st["dtype"])
    if op == "transpose":
        return capi.mxfp4_dequantize(capi.mxfp4_quantize_transposed(st["x"]), dtype=st["dtype"])
    if op == "linear":
        w = capi.Mxfp4(st["codes"], st["scales"], st["N"], st["K"])
        return capi.mxfp4_linear(st["x"], w)
    if op == "experts":
        w = capi.Mxfp4(st["codes"], st["scales"], st["E"] * st["N"], st["K"])
        return capi.mxfp4_linear(st["x"], w, perm=st["perm"], expert_offsets=st["offsets"],
                                 expert_counts=st["counts"], row_weight=st["row_weight"], out=st["y"])
    if op == "weight_grad":
        return capi.mxfp4_matmul(capi.mxfp4_quantize_transposed(st["dy"]), capi.mxfp4_quantize_transposed(st["x"]),
                                 out_dtype=torch.float32)
    b = capi.moe_balance_loss(st["logits"], st["topk_idx"], st["coeff"], score=st["score"], token_mask=st["mask"],
                              seq_offsets=st["seq_offsets"])
    d = capi.moe_balance_loss_backward(st["logits"], b, st["grad_loss"])
    return dict(loss=b.loss, counts=b.counts, probs=b.probs, dlogits=d)


# ---------------------------------------------------------------------------
# 64-bit values, from the definitions
# ---------------------------------------------------------------------------

def _power(n):
    return torch.ldexp(torch.ones_like(n, dtype=torch.float64), n)


def _exact_quantized(x):
    """The MXFP4 values of a matrix's rows: each element to the nearest
    multiple of its binade's spacing under the block's power of two."""
    rows, cols = x.shape
    n = -(-cols // 32)
    buf = torch.zeros((rows, n * 32), dtype=torch.float64, device=x.device)
    buf[:, :cols] = x
    buf = buf.view(rows, n, 32)
    top = buf.abs().max(dim=2, keepdim=True).values
    # frexp: top = m 2^e with m in [1/2, 1), so floor(log2 top) = e - 1
    scale = _power((torch.frexp(top).exponent - 3).clamp(min=-127).masked_fill(top == 0, -127))
    v = buf / scale
    step = _power(torch.frexp(v.abs().clamp(1.0, 6.0)).exponent - 2)
    v = (torch.round(v / step) * step).clamp(-6.0, 6.0)
    return (v * scale).view(rows, n * 32)


def _exact_weights(codes, scales):
    rows, half = codes.shape
    lo, hi = codes.long() % 16, codes.long() // 16
    c = torch.stack((lo, hi), dim=-1).view(rows, half * 2)
    m = c % 8
    mag = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * _power(m // 2 - 1))
    mag = torch.where(c >= 8, -mag, mag)
    nb = half // 16
    groups = -(-nb // 4)
    # atoms [row tile, group][32 rows][4 quarters][4 blocks] -> rows x blocks
    s = scales.view(-1, groups, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, groups * 4)[:rows, :nb]
    return mag * _power(s.to(torch.int32) - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        return _exact_quantized(st["x"])[:, :st["cols"]]
    if op == "transpose":
        return _exact_quantized(st["x"].t())[:, :st["rows"]]
    if op == "linear":
        return torch.matmul(_exact_quantized(st["x"]), _exact_weights(st["codes"], st["scales"]).t())
    if op == "experts":
        x, w = _exact_quantized(st["x"]), _exact_weights(st["codes"], st["scales"])
        out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        offsets, counts, N = st["offsets"].tolist(), st["counts"].tolist(), st["N"]
        for e in range(st["E"]):
            at = slice(offsets[e], offsets[e] + counts[e])
            y = x[st["perm"][at].long()] @ w[e * N:(e + 1) * N].t()
            out[at] = y * st["row_weight"][at].double()[:, None]
        return out
    if op == "weight_grad":
        return torch.matmul(_exact_quantized(st["dy"].t()), _exact_quantized(st["x"].t()).t())
    return _exact_balance(st)


def _exact_balance(st):
    """Sequence by sequence, the gradient by the chain rule of the log scores:
    with p = softmax(z), dL/dz = g p (f - <f, p>), z the logits or log sigma
    (whose derivative is sigma of the negated logit)."""
    logits = st["logits"].double()
    T, E = logits.shape
    k, S = st["k"], st["S"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
    z = logits if st["score"] == "softmax" else torch.nn.functional.logsigmoid(logits)
    dz = torch.ones_like(logits) if st["score"] == "softmax" else torch.sigmoid(-logits)
    p = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))
    counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    probs = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    d = torch.zeros_like(logits)
    bounds = st["seq_offsets"].tolist()
    full = [s for s in range(S) if int(keep[bounds[s]:bounds[s + 1]].sum()) > 0]
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    for s in full:
        t = torch.arange(bounds[s], bounds[s + 1], device="cuda")[keep[bounds[s]:bounds[s + 1]]]
        n = t.numel()
        counts[s] = torch.bincount(st["topk_idx"][t].long().reshape(-1), minlength=E).to(torch.int32)
        probs[s] = p[t].sum(dim=0) / n
        f = counts[s].double() * E / (k * n)
        loss += st["coeff"] / len(full) * (f @ probs[s])
        g = st["grad_loss"].double() * st["coeff"] / (len(full) * n)
        d[t] = g * p[t] * (f - (p[t] @ f)[:, None]) * dz[t]
    return dict(loss=loss, counts=counts, probs=probs, dlogits=d)
