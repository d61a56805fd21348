"""What is measured of the block's 8-bit weights: the quantiser, the dense
skinny product and the whole decode MoE layer, each beside its plain form.

Weights are OCP e4m3 with one fp32 scale for each 128 x 128 block, activations
bf16 or e4m3 with one scale for each 128 columns of a row.  Sizes follow the
decode block's own workloads (hidden size 7168, 384 experts, top-8, expert
rows of 128 or 256, batch 1 to 64) and generic ones around them.
"""
import math

import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The activations of one decode step at batch 8, ahead of an 8-bit product: latency.
        {"name": "quantize_rows_b8", "op": "quantize", "layout": "rows", "n": 1, "rows": 8, "cols": 7168, "dtype": "bf16"},
        # An odd number of fp32 rows whose last scale group is short.
        {"name": "quantize_rows_odd_f32", "op": "quantize", "layout": "rows", "n": 1, "rows": 61, "cols": 1040, "dtype": "f32"},
        # One rank's gate/up weights of 64 experts at load time: a stream of half a gigabyte.
        {"name": "quantize_blocks_experts", "op": "quantize", "layout": "blocks", "n": 128, "rows": 256, "cols": 7168, "dtype": "bf16"},
        # Attention output projection with its residual at batch 1: the smallest decode call.
        {"name": "gemm_b1_residual", "op": "gemm", "B": 1, "N": 7168, "K": 2048, "x": "bf16", "residual": True, "out": "bf16"},
        # Attention input projection of one rank at batch 8, bf16 activations.
        {"name": "gemm_b8", "op": "gemm", "B": 8, "N": 2304, "K": 7168, "x": "bf16", "residual": False, "out": "bf16"},
        # A square projection over a small batch, both operands in 8 bits.
        {"name": "gemm_b5_e4m3", "op": "gemm", "B": 5, "N": 7168, "K": 7168, "x": "e4m3", "residual": False, "out": "bf16"},
        # Odd batch, odd rows and a short last block on both axes, fp32 out.
        {"name": "gemm_b33_odd", "op": "gemm", "B": 33, "N": 1001, "K": 1040, "x": "bf16", "residual": False, "out": "f32"},
        # The largest batch of the decode range over a square projection, both operands in 8 bits.
        {"name": "gemm_b64_e4m3", "op": "gemm", "B": 64, "N": 7168, "K": 7168, "x": "e4m3", "residual": True, "out": "bf16"},
        # A small layer at batch 2, shorter scale blocks than 128 in the experts: launches and waits count.
        {"name": "moe_small_b2", "op": "moe", "B": 2, "d": 1024, "E": 32, "k": 4, "I": 64, "Is": 64, "routing": "plain"},
        # One rank's shard of a 16-way split at batch 1: one sequence being decoded.
        {"name": "moe_tp16_b1", "op": "moe", "B": 1, "d": 7168, "E": 384, "k": 8, "I": 128, "Is": 128, "routing": "plain"},
        # The same shard at batch 8, noisy routing: nearly every choice another expert.
        {"name": "moe_tp16_b8", "op": "moe", "B": 8, "d": 7168, "E": 384, "k": 8, "I": 128, "Is": 128, "routing": "gumbel"},
        # One rank's shard of an 8-way split at batch 64, a few experts much in demand.
        {"name": "moe_tp8_b64", "op": "moe", "B": 64, "d": 7168, "E": 384, "k": 8, "I": 256, "Is": 256, "routing": "zipf"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "moe", "moe"])
    if op == "quantize":
        layout = rng.choice(["rows", "blocks"])
        cols = 16 * _log(rng, 8, 512)
        rows = _log(rng, 1, 64) if layout == "rows" else _log(rng, 32, 8192)
        n = 1 if layout == "rows" else _log(rng, 1, max(1, min(128, 128 * 256 * 7168 // (rows * cols))))
        return {"op": op, "layout": layout, "n": n, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"])}
    B = _log(rng, 1, 64)
    if op == "gemm":
        K = 16 * _log(rng, 8, 512)
        N = _log(rng, 16, max(16, min(12288, 7168 * 7168 // K)))
        return {"op": op, "B": B, "N": N, "K": K, "x": rng.choice(["bf16", "e4m3"]),
                "residual": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "f32"])}
    E = _log(rng, 16, 384)
    k = rng.randint(1, min(E, 16, 512 // B))
    return {"op": op, "B": B, "d": 32 * rng.randint(16, 224), "E": E, "k": k, "I": 32 * rng.randint(1, 8),
            "Is": 32 * rng.randint(0, 8), "routing": rng.choice(["plain", "gumbel", "zipf"])}


# ---- inputs ------------------------------------------------------------------


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _codes(gen, shape):
    """e4m3 codes as the quantiser leaves them of normal weights: the largest of a 16384-value block, about 4.2
    standard deviations, lies near 448.  Drawn in pieces, so that no fp32 copy of all experts is held."""
    q = torch.empty(shape, dtype=E4M3, device="cuda")
    flat = q.view(-1, shape[-1])
    step = max(1, (1 << 28) // shape[-1])
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_((torch.randn(part.shape, generator=gen, device="cuda") * 107.0).clamp_(-E4M3_MAX, E4M3_MAX))
    return q


def _scales(gen, shape, fan_in):
    return (1.0 + 0.3 * torch.rand(shape, generator=gen, device="cuda")) * (fan_in ** -0.5 / 107.0)


def _bias(case, gen):
    """Added to the router's logits: none, Gumbel noise for each token, or a Zipf(1.1) log-prior over the experts."""
    B, E = case["B"], case["E"]
    if case["routing"] == "gumbel":
        u = torch.rand((B, E), generator=gen, device="cuda", dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
        return (-(-u.log()).log()).float(), E
    if case["routing"] == "zipf":
        rank = torch.randperm(E, generator=gen, device="cuda") + 1
        return -1.1 * rank.float().log(), 0
    return None, 0


def _clear_tokens(case, gen, Wr):
    """Activations and bias of B tokens whose k-th and next logits are not within 1e-3 of each other (a pair that
    close is split by the order of a sum): four times as many are drawn, and the first clear ones kept."""
    B, d, E, k = case["B"], case["d"], case["E"], case["k"]
    many = dict(case, B=4 * B + 16)
    X = torch.randn((many["B"], d), generator=gen, device="cuda").to(torch.bfloat16)
    bias, ld = _bias(many, gen)
    if k < E:
        logits = X.double() @ Wr.double().t()
        if bias is not None:
            logits = logits + bias.double()
        top = logits.topk(k + 1, dim=1).values
        keep = ((top[:, k - 1] - top[:, k]) < 1e-3).long().argsort(stable=True)[:B]
    else:
        keep = torch.arange(B, device="cuda")
    return X[keep].contiguous(), bias if bias is None or ld == 0 else bias[keep].contiguous(), ld


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        X = torch.randn((n, rows, cols), generator=gen, device="cuda")
        # rows of different sizes, as activations and weights have them
        X *= torch.exp2(2.0 * torch.randn((n, rows, 1), generator=gen, device="cuda"))
        s["X"] = X.to(DTYPES[case["dtype"]])
        r = rows if case["layout"] == "rows" else _blocks(rows)
        s["Q"] = torch.empty((n, rows, cols), dtype=E4M3, device="cuda")
        s["scale"] = torch.empty((n, r, _blocks(cols)), dtype=torch.float32, device="cuda")
        return s
    if case["op"] == "gemm":
        B, N, K = case["B"], case["N"], case["K"]
        s["W"], s["Ws"] = _codes(gen, (N, K)), _scales(gen, (_blocks(N), _blocks(K)), K)
        if case["x"] == "e4m3":
            # unit-variance activations: the largest of 128 lies near 2.7 standard deviations
            s["X"] = (torch.randn((B, K), generator=gen, device="cuda") * 128.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
            s["Xs"] = torch.exp2(torch.randint(-8, -5, (B, _blocks(K)), generator=gen, device="cuda").float())
        else:
            s["X"], s["Xs"] = torch.randn((B, K), generator=gen, device="cuda").to(torch.bfloat16), None
        s["R"] = torch.randn((B, N), generator=gen, device="cuda").to(torch.bfloat16) if case["residual"] else None
        s["Y"] = torch.empty((B, N), dtype=DTYPES[case["out"]], device="cuda")
        if own:
            from moe_block_skinny_amd import binding as mb
            s["weight"] = mb.Fp8Weight(s["W"], s["Ws"])
            need = mb.workspace_bytes(mb.OP_SKINNY_GEMM_FP8, mb.DT_E4M3 if s["Xs"] is not None else mb.DT_BF16,
                                      B=B, N=N, K=K)
            s["ws"] = mb.workspace(need) if need else None
        return s
    B, d, E, k, I, Is = (case[q] for q in ("B", "d", "E", "k", "I", "Is"))
    s["Wr"] = (torch.randn((E, d), generator=gen, device="cuda") * d ** -0.5).to(torch.bfloat16)
    s["X"], s["bias"], s["bias_ld"] = _clear_tokens(case, gen, s["Wr"])
    # one row of scales for each 128 gate rows, then for each 128 up rows
    s["W13"], s["s13"] = _codes(gen, (E, 2 * I, d)), _scales(gen, (E, 2 * _blocks(I), _blocks(d)), d)
    s["W2"], s["s2"] = _codes(gen, (E, d, I)), _scales(gen, (E, _blocks(d), _blocks(I)), I)
    s["Ws13"] = s["ss13"] = s["Ws2"] = s["ss2"] = None
    if Is:
        s["Ws13"], s["ss13"] = _codes(gen, (2 * Is, d)), _scales(gen, (2 * _blocks(Is), _blocks(d)), d)
        s["Ws2"], s["ss2"] = _codes(gen, (d, Is)), _scales(gen, (_blocks(d), _blocks(Is)), Is)
    s["out"] = torch.empty((B, d), dtype=torch.bfloat16, device="cuda")
    s["ids"] = torch.empty((B, k), dtype=torch.int32, device="cuda")
    s["w"] = torch.empty((B, k), dtype=torch.float32, device="cuda")
    if own:
        from moe_block_skinny_amd import binding as mb
        s["experts"] = mb.Fp8Experts(s["W13"], s["s13"], s["W2"], s["s2"], s["Ws13"], s["ss13"], s["Ws2"], s["ss2"])
        s["ws"] = mb.workspace(mb.workspace_bytes(mb.OP_BLOCK_FP8, mb.DT_BF16, B=B, d=d, E=E, k=k, I=I, Is=Is))
    return s


# ---- one pass ----------------------------------------------------------------


def run(s):
    return {"quantize": _quantize, "gemm": _gemm, "moe": _moe}[s["op"]](s)


def _quantize(s):
    if own:
        from moe_block_skinny_amd import binding as mb
        mb.moe_quantize_fp8(s["X"], s["Q"], s["scale"], s["layout"])
        return s["Q"], s["scale"]
    X = s["X"].float()
    n, rows, cols = X.shape
    tall = 1 if s["layout"] == "rows" else BLOCK
    r, c = (rows + tall - 1) // tall, _blocks(cols)
    pad = torch.nn.functional.pad(X, (0, c * BLOCK - cols, 0, r * tall - rows)).view(n, r, tall, c, BLOCK)
    largest = pad.abs().amax(dim=(2, 4))
    # the smallest power of two that brings the block within 448: m 2^e = largest / 448, 1/2 <= m < 1
    m, e = torch.frexp(largest.double() / E4M3_MAX)
    scale = torch.where(largest > 0, torch.exp2((e - (m == 0.5).int()).clamp_min(-126).float()), 1.0)
    Q = (pad / scale[:, :, None, :, None]).to(E4M3).view(n, r * tall, c * BLOCK)
    return Q[:, :rows, :cols].contiguous(), scale


def _spread(scale, rows, cols):
    """A block's scale for each of its values."""
    wide = scale.repeat_interleave(BLOCK, dim=-1)[..., :cols]
    return wide.repeat_interleave(BLOCK, dim=-2)[..., :rows, :]


def _gemm(s):
    if own:
        from moe_block_skinny_amd import binding as mb
        mb.skinny_gemm_fp8(s["X"], s["weight"], s["Y"], x_scale=s["Xs"], R=s["R"], ws=s["ws"])
        return s["Y"]
    W = s["W"].float() * _spread(s["Ws"], s["N"], s["K"])
    X = s["X"].float()
    if s["Xs"] is not None:
        X = X * s["Xs"].repeat_interleave(BLOCK, dim=1)[:, :s["K"]]
    Y = X @ W.t()
    if s["R"] is not None:
        Y = Y + s["R"].float()
    return Y.to(s["Y"].dtype)


def _swiglu(a, I):
    g, u = a[..., :I], a[..., I:]
    return g / (1.0 + torch.exp(-g)) * u


def _spread13(scale, I, d):
    """Gate and up rows have their own blocks."""
    halves = scale.view(scale.shape[:-2] + (2, _blocks(I), scale.shape[-1]))
    return _spread(halves, I, d).reshape(scale.shape[:-2] + (2 * I, d))


def _moe(s):
    if own:
        from moe_block_skinny_amd import binding as mb
        mb.moe_block_fp8(s["X"], s["Wr"], s["k"], s["experts"], s["out"], s["ws"], bias=s["bias"],
                         bias_ld=s["bias_ld"], topk_ids=s["ids"], topk_w=s["w"])
        return {"out": s["out"], "ids": s["ids"], "weights": s["w"]}
    B, d, k, I, Is = (s[q] for q in ("B", "d", "k", "I", "Is"))
    X = s["X"].float()
    logits = X @ s["Wr"].float().t()
    if s["bias"] is not None:
        logits = logits + s["bias"]
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(dim=1).values
    chosen = logits.gather(1, ids)
    w = torch.exp(chosen - chosen.amax(dim=1, keepdim=True))
    w = w / w.sum(dim=1, keepdim=True)
    e = ids.reshape(-1)
    W13 = s["W13"].view(torch.uint8)[e].view(E4M3).float() * _spread13(s["s13"][e], I, d)
    x = X.repeat_interleave(k, dim=0).unsqueeze(2)
    h = _swiglu(torch.bmm(W13, x).squeeze(2), I)
    W2 = s["W2"].view(torch.uint8)[e].view(E4M3).float() * _spread(s["s2"][e], d, I)
    y = torch.bmm(W2, h.unsqueeze(2)).view(B, k, d)
    out = (w.unsqueeze(2) * y).sum(dim=1)
    if Is:
        hs = _swiglu(X @ (s["Ws13"].float() * _spread13(s["ss13"], Is, d)).t(), Is)
        out = out + hs @ (s["Ws2"].float() * _spread(s["ss2"], d, Is)).t()
    return {"out": out.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": w}


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    if case["op"] == "quantize":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        r = rows if case["layout"] == "rows" else _blocks(rows)
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * rows * cols * (size + 1) + 4 * n * r * _blocks(cols), "flops": 2 * n * rows * cols}
    if case["op"] == "gemm":
        B, N, K = case["B"], case["N"], case["K"]
        x = B * K * 2 if case["x"] == "bf16" else B * (K + 4 * _blocks(K))
        y = B * N * ((2 if case["out"] == "bf16" else 4) + (2 if case["residual"] else 0))
        return {"bytes": N * K + 4 * _blocks(N) * _blocks(K) + x + y, "flops": 2 * B * N * K}
    B, d, E, k, I, Is = (case[q] for q in ("B", "d", "E", "k", "I", "Is"))
    # experts that at least one token chooses: the mean over 16 draws of logits as the routing has them
    gen = torch.Generator().manual_seed(1)
    logits = torch.randn((16, B, E), generator=gen)
    if case["routing"] == "gumbel":
        logits -= torch.empty((16, B, E)).exponential_(generator=gen).log()
    if case["routing"] == "zipf":
        logits -= 1.1 * torch.arange(1, E + 1).float().log()
    chosen = torch.zeros((16, E)).scatter_(1, logits.topk(k, dim=2).indices.view(16, -1), 1.0)
    n = float(chosen.sum(dim=1).mean())

    def expert(i):
        return 3 * i * d + 4 * (2 * _blocks(i) * _blocks(d) + _blocks(d) * _blocks(i))

    size = n * expert(I) + (expert(Is) if Is else 0) + 2 * E * d + 4 * B * d + 8 * B * k
    size += {"plain": 0, "gumbel": 4 * B * E, "zipf": 4 * E}[case["routing"]]
    return {"bytes": size, "flops": 2 * B * d * (E + 3 * (k * I + Is))}


# ---- the same in 64 bits ---------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "gemm": _exact_gemm, "moe": _exact_moe}[case["op"]](s)


def _exact_quantize(s):
    n, rows, cols = s["X"].shape
    tall = 1 if s["layout"] == "rows" else BLOCK
    Q = torch.empty((n, rows, cols), dtype=torch.float64, device="cuda")
    scale = torch.empty(s["scale"].shape, dtype=torch.float64, device="cuda")
    for c in range(_blocks(cols)):
        col = slice(c * BLOCK, min(cols, (c + 1) * BLOCK))
        x = s["X"][:, :, col].double()
        widest = x.abs().amax(dim=2)
        for r in range(0, rows, tall) if tall > 1 else [slice(0, rows)]:
            row = r if tall == 1 else slice(r, min(rows, r + tall))
            big = widest[:, row] if tall == 1 else widest[:, row].amax(dim=1, keepdim=True)
            p = torch.exp2(torch.ceil(torch.log2(big / E4M3_MAX)))
            p = torch.where(p / 2 >= big / E4M3_MAX, p / 2, torch.where(p < big / E4M3_MAX, p * 2, p))
            p = torch.where(big > 0, p.clamp_min(2.0 ** -126), 1.0)
            v = x[:, row] / p.unsqueeze(2)
            # the grid of e4m3 at v: 3 bits after the leading one, at least 2^-9
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            Q[:, row, col] = torch.round(v / step) * step
            if tall == 1:
                scale[:, :, c] = p
            else:
                scale[:, r // tall, c] = p[:, 0]
    return Q, scale


def _exact_product(X, W, scale, rows_of=None):
    """X W^T in 64 bits, block after block: scale[i][j] is that of rows i * 128 .. and columns j * 128 .. of W."""
    N, K = W.shape
    Y = torch.zeros((X.shape[0], N), dtype=torch.float64, device="cuda")
    for j in range(_blocks(K)):
        col = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
        part = X[:, col] @ W[:, col].double().t().contiguous()
        Y += part * scale[:, j].double()[torch.arange(N, device="cuda") // BLOCK if rows_of is None else rows_of]
    return Y


def _exact_gemm(s):
    X = s["X"].double()
    if s["Xs"] is not None:
        X = X * s["Xs"].double()[:, torch.arange(s["K"], device="cuda") // BLOCK]
    Y = _exact_product(X, s["W"], s["Ws"])
    return Y if s["R"] is None else Y + s["R"].double()


def _exact_expert(X, W13, s13, W2, s2):
    I = W2.shape[1]
    i = torch.arange(I, device="cuda") // BLOCK
    a = _exact_product(X, W13, s13, torch.cat([i, i + _blocks(I)]))
    z = a[:, :I]
    return _exact_product(z * torch.sigmoid(z) * a[:, I:], W2, s2)


def _exact_moe(s):
    B, k = s["B"], s["k"]
    X = s["X"].double()
    logits = X @ s["Wr"].double().t().contiguous()
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    ids = torch.topk(logits, k, dim=1).indices.sort(dim=1).values
    w = torch.softmax(torch.gather(logits, 1, ids), dim=1)
    out = torch.zeros((B, s["d"]), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        out[t] += w[t, j].unsqueeze(1) * _exact_expert(X[t], s["W13"][e], s["s13"][e], s["W2"][e], s["s2"][e])
    if s["Is"]:
        out += _exact_expert(X, s["Ws13"], s["ss13"], s["Ws2"], s["ss2"])
    return {"out": out, "ids": ids.to(torch.int32), "weights": w}
