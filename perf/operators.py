"""What the 4-bit weight operators and the embedding lookup with its gradient compute, in plain torch, and the cases
they are measured on.

    quantise   W [N, K] to packed 4-bit codes with one scale (and zero point) per group, and back to values
    matvec     y = x W^T for 1 to 32 tokens x [M, K], W in that format
    lookup     rows of a table (bf16, fp32, e4m3 with 1x128 scales, or 4-bit) times a factor
    gradient   of the lookup, dense over the table

Format of a 4-bit matrix: codes 0..15, two to a byte (even k in the low nibble), scale [N, ceil(K / group)] in fp32 or
bf16, zero uint8 of the same shape or none (then 8): value = scale * (code - zero).
"""
import torch
import torch.nn.functional as F

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}

# The largest listed work of each operator; drawn cases stay below it.
MOST_WEIGHTS = 131072 * 5120  # elements of a 4-bit matrix that a product reads
MOST_QUANT = 5120 * 8192      # elements that a quantisation reads
MOST_TOKENS = 16640
MOST_TABLE = 131072 * 5120    # elements of a token table


def listed():
    return [
        # a small projection quantised with zero points in fine groups, from fp32 master weights
        {"name": "quantise_small", "op": "quantise", "N": 1024, "K": 4096, "group": 32, "x": "f32", "scale": "f32", "asym": True},
        # a matrix whose rows end inside a group and inside a byte, bf16 scales
        {"name": "quantise_ragged", "op": "quantise", "N": 2085, "K": 4099, "group": 64, "x": "bf16", "scale": "bf16", "asym": False},
        # the weight of the headline layer
        {"name": "quantise_layer", "op": "quantise", "N": 5120, "K": 8192, "group": 128, "x": "bf16", "scale": "f32", "asym": False},
        # one token through a small projection: latency
        {"name": "matvec_token", "op": "matvec", "M": 1, "N": 1024, "K": 4096, "group": 128, "x": "bf16", "scale": "bf16", "asym": False, "bias": False},
        # a decoding batch through the layer of the small-M sweep, zero points and a bias
        {"name": "matvec_batch", "op": "matvec", "M": 8, "N": 7168, "K": 2048, "group": 64, "x": "bf16", "scale": "bf16", "asym": True, "bias": True},
        # fp32 activations, odd output count, a last group of 16
        {"name": "matvec_f32", "op": "matvec", "M": 5, "N": 8191, "K": 8208, "group": 32, "x": "f32", "scale": "f32", "asym": False, "bias": False},
        # the output head of a large vocabulary for sixteen sequences
        {"name": "matvec_head", "op": "matvec", "M": 16, "N": 131072, "K": 5120, "group": 128, "x": "bf16", "scale": "bf16", "asym": False, "bias": False},
        # decoding: the rows of eight tokens from a 4-bit table
        {"name": "lookup_decode", "op": "lookup", "T": 8, "V": 131072, "D": 5120, "table": "int4", "group": 128, "out": "bf16"},
        # a training batch's rows from a bf16 table
        {"name": "lookup_batch", "op": "lookup", "T": 16640, "V": 131072, "D": 5120, "table": "bf16", "group": 128, "out": "bf16"},
        # a short batch on a small vocabulary, odd row length, bf16 gradient table
        {"name": "gradient_small", "op": "gradient", "T": 255, "V": 7168, "D": 1001, "grad": "f32", "out": "bf16", "pad": 0.0},
        # sequences padded to one length: an eighth of the tokens name the padding row
        {"name": "gradient_padded", "op": "gradient", "T": 8192, "V": 32768, "D": 2048, "grad": "bf16", "out": "f32", "pad": 0.125},
        # the training batch of lookup_batch
        {"name": "gradient_batch", "op": "gradient", "T": 16640, "V": 131072, "D": 5120, "grad": "bf16", "out": "f32", "pad": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantise", "matvec", "lookup", "gradient"])
    group = rng.choice([32, 64, 128])
    if op == "quantise":
        K = _log(rng, 100, 16384)
        return {"op": op, "N": _log(rng, 64, min(16384, MOST_QUANT // K)), "K": K, "group": group, "x": rng.choice(["bf16", "f32"]),
                "scale": rng.choice(["bf16", "f32"]), "asym": rng.random() < 0.5}
    if op == "matvec":
        K = 2 * _log(rng, 64, 8192)
        return {"op": op, "M": _log(rng, 1, 32), "N": _log(rng, 64, min(131072, MOST_WEIGHTS // K // 4)), "K": K, "group": group,
                "x": rng.choice(["bf16", "bf16", "f32"]), "scale": rng.choice(["bf16", "f32"]), "asym": rng.random() < 0.5,
                "bias": rng.random() < 0.5}
    D = _log(rng, 64, 8192)
    V = _log(rng, 256, min(262144, MOST_TABLE // D))
    T = _log(rng, 1, MOST_TOKENS)
    if op == "lookup":
        table = rng.choice(["bf16", "f32", "e4m3", "int4"])
        return {"op": op, "T": T, "V": V, "D": D + D % 2 if table == "int4" else D, "table": table, "group": group,
                "out": rng.choice(["bf16", "f32"])}
    return {"op": op, "T": T, "V": V, "D": D, "grad": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
            "pad": rng.choice([0.0, 0.25])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pad_rows(shape, dtype):
    """Empty [rows, cols] whose rows start on 16-byte boundaries, as an aligned allocation keeps them."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty(shape[0], -(-shape[1] // per) * per, dtype=dtype, device=DEVICE)[:, :shape[1]]


def _codes(gen, N, K, group, scale_dtype, asym):
    """A 4-bit matrix as a quantised weight is: codes near normal, scales of one magnitude."""
    q = _pad_rows((N, -(-K // 2)), torch.uint8)
    step = max(1, (1 << 26) // max(1, K))
    for r in range(0, N, step):  # in bands, so that the draws stay small
        w = torch.randn(min(step, N - r), 2 * q.shape[1], generator=gen, device=DEVICE)
        c = (w * 2.4 + 8).round().clamp(1, 15).to(torch.uint8).view(w.shape[0], -1, 2)
        q[r:r + w.shape[0]] = c[..., 0] | (c[..., 1] << 4)
    G = -(-K // group)
    s = (torch.rand(N, G, generator=gen, device=DEVICE) + 0.5).mul_(0.008).to(scale_dtype)
    z = torch.randint(5, 11, (N, G), generator=gen, device=DEVICE).to(torch.uint8) if asym else None
    return q, s, z


def _tokens(gen, T, V):
    """Token numbers with the frequencies of text: the k-th most frequent about 1/k, scattered over the vocabulary."""
    k = torch.pow(torch.tensor(float(V), device=DEVICE), torch.rand(T, generator=gen, device=DEVICE)).long().clamp_(1, V) - 1
    return (k * 40503 + 17) % V


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantise":
        x = torch.randn(case["N"], case["K"], generator=gen, device=DEVICE)
        x = torch.where(torch.rand(x.shape, generator=gen, device=DEVICE) < 0.01, x * 8, x) * 0.02
        s["w"] = _pad_rows(x.shape, DTYPES[case["x"]]).copy_(x)
    elif case["op"] == "matvec":
        s["q"], s["s"], s["z"] = _codes(gen, case["N"], case["K"], case["group"], DTYPES[case["scale"]], case["asym"])
        s["x"] = torch.randn(case["M"], case["K"], generator=gen, device=DEVICE).to(DTYPES[case["x"]])
        s["b"] = torch.randn(case["N"], generator=gen, device=DEVICE) if case["bias"] else None
    elif case["op"] == "lookup":
        V, D = case["V"], case["D"]
        s["tokens"] = _tokens(gen, case["T"], V)
        s["alpha"] = float(D) ** 0.5
        s["s"] = s["z"] = None
        if case["table"] == "int4":
            s["t"], s["s"], s["z"] = _codes(gen, V, D, case["group"], torch.float32, False)
        elif case["table"] == "e4m3":
            s["t"] = _pad_rows((V, D), torch.uint8)
            s["t"].copy_((torch.randn(V, D, generator=gen, device=DEVICE) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            s["s"] = (torch.rand(V, -(-D // 128), generator=gen, device=DEVICE) + 0.5) * 2e-4
        else:
            s["t"] = _pad_rows((V, D), DTYPES[case["table"]])
            step = max(1, (1 << 27) // D)
            for r in range(0, V, step):
                s["t"][r:r + step] = torch.randn(min(step, V - r), D, generator=gen, device=DEVICE) * 0.02
    else:
        s["tokens"] = _tokens(gen, case["T"], case["V"])
        s["pad_row"] = 3 if case["pad"] else None
        if case["pad"]:
            s["tokens"] = torch.where(torch.rand(case["T"], generator=gen, device=DEVICE) < case["pad"], 3, s["tokens"])
        g = torch.randn(case["T"], case["D"], generator=gen, device=DEVICE) * 1e-3
        s["g"] = _pad_rows(g.shape, DTYPES[case["grad"]]).copy_(g)
        s["alpha"] = float(case["D"]) ** 0.5
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _unpack(q, s, z, K, group):
    """Values of a 4-bit matrix, fp32 [rows, K]."""
    c = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], -1)[:, :K].float()
    each = lambda v: v.float().repeat_interleave(group, 1)[:, :K]  # noqa: E731
    return (c - (8.0 if z is None else each(z))) * each(s)


def _quantise(w, group, scale_dtype, asym):
    N, K = w.shape
    x = F.pad(w.float(), (0, -K % group)).view(N, -1, group)
    # the divisors are tensors: a quotient by a Python number is taken by way of its reciprocal
    if asym:
        lo, hi, n = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0), x.new_full((), 15.0)
        s = (hi / n - lo / n).to(scale_dtype)
    else:
        s = (x.abs().amax(-1) / x.new_full((), 7.0)).to(scale_dtype)
    s = torch.where(s == 0, torch.ones_like(s), s)
    each = s.float()
    c = torch.round(x / each[..., None])
    if asym:
        z = torch.round(-lo / each).clamp(0, 15)
        v = (c + z[..., None]).clamp(0, 15) - z[..., None]
        z = z.to(torch.uint8)
    else:
        v, z = c.clamp(-8, 7), None
    return (v * each[..., None]).view(N, -1)[:, :K].to(w.dtype), s, z


def _plain(s):
    if s["op"] == "quantise":
        v, sc, z = _quantise(s["w"], s["group"], DTYPES[s["scale"]], s["asym"])
        return {"values": v, "scale": sc, "zero": z}
    if s["op"] == "matvec":
        y = s["x"].float() @ _unpack(s["q"], s["s"], s["z"], s["K"], s["group"]).t()
        return {"y": (y if s["b"] is None else y + s["b"]).to(s["x"].dtype)}
    if s["op"] == "lookup":
        t = s["tokens"]
        rows = s["t"][t]
        if s["table"] == "int4":
            rows = _unpack(rows, s["s"][t], None, s["D"], s["group"])
        elif s["table"] == "e4m3":
            rows = rows.view(torch.float8_e4m3fn).float() * s["s"][t].repeat_interleave(128, 1)[:, :s["D"]]
        return {"rows": (rows.float() * s["alpha"]).to(DTYPES[s["out"]])}
    t, g = s["tokens"], s["g"].float() * s["alpha"]
    if s["pad_row"] is not None:
        g = g * (t != s["pad_row"])[:, None]
    d = torch.zeros(s["V"], s["D"], device=g.device)
    return {"table": d.index_add_(0, t, g).to(DTYPES[s["out"]])}


def _own(s):
    import int8_gemm_b200 as bs

    if s["op"] == "quantise":
        q, sc, z = bs.bs_quantize_int4(s["w"], group=s["group"], scale_dtype=DTYPES[s["scale"]], asymmetric=s["asym"])
        return {"values": bs.bs_dequantize_int4(q, sc, z, K=s["K"], group=s["group"], out_dtype=s["w"].dtype), "scale": sc, "zero": z}
    if s["op"] == "matvec":
        return {"y": bs.bs_gemv_int4(s["x"], s["q"], s["s"], s["z"], s["b"], group=s["group"], out_dtype=s["x"].dtype)}
    if s["op"] == "lookup":
        fmt = s["table"] if s["table"] in ("int4", "e4m3") else "dense"
        return {"rows": bs.bs_embedding(s["tokens"], s["t"], s["s"], s["z"], format=fmt, dim=s["D"], group=s["group"], alpha=s["alpha"],
                                        out_dtype=DTYPES[s["out"]])}
    return {"table": bs.bs_embedding_grad(s["tokens"], s["g"], s["V"], alpha=s["alpha"], padding_idx=s["pad_row"],
                                          out_dtype=DTYPES[s["out"]])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] in ("quantise", "matvec"):
        N, K = case["N"], case["K"]
        q4 = N * -(-K // 2) + N * -(-K // case["group"]) * (BYTES[case["scale"]] + (1 if case["asym"] else 0))
        if case["op"] == "quantise":  # read, coded, read back as codes, written as values
            return {"bytes": 2 * q4 + 2 * N * K * BYTES[case["x"]], "flops": 4 * N * K}
        M = case["M"]
        return {"bytes": q4 + M * (N + K) * BYTES[case["x"]] + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, V, D = case["T"], case["V"], case["D"]
    if case["op"] == "lookup":
        # every row that is named is read once: with text's frequencies about T of them, at most V
        row = {"bf16": 2 * D, "f32": 4 * D, "e4m3": D + 4 * -(-D // 128), "int4": D // 2 + 4 * -(-D // case["group"])}[case["table"]]
        return {"bytes": min(T, V) * row + T * (8 + D * BYTES[case["out"]]), "flops": T * D}
    return {"bytes": T * (8 + D * BYTES[case["grad"]]) + V * D * BYTES[case["out"]], "flops": T * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        # scales and quotients are fp32 numbers by definition (codes decide on them, ties to even): each is its 64-bit
        # value rounded once
        w, g = s["w"].double(), case["group"]
        f32 = lambda v: v.float().double()  # noqa: E731
        N, K = w.shape
        values, scales, zeros = torch.empty_like(w), [], []
        for k in range(0, K, g):
            x = w[:, k:k + g]
            if case["asym"]:
                lo, hi = x.min(1).values.clamp(max=0), x.max(1).values.clamp(min=0)
                sc = (f32(hi / 15) - f32(lo / 15)).float().to(DTYPES[case["scale"]]).double()
            else:
                sc = (x.abs().max(1).values / 7).float().to(DTYPES[case["scale"]]).double()
            sc[sc == 0] = 1
            if case["asym"]:
                z = torch.clamp(torch.round(f32(-lo / sc)), 0, 15)
                zeros.append(z)
            low, high = (-z[:, None], 15 - z[:, None]) if case["asym"] else (torch.full_like(sc, -8)[:, None], torch.full_like(sc, 7)[:, None])
            values[:, k:k + g] = torch.minimum(torch.maximum(torch.round(f32(x / sc[:, None])), low), high) * sc[:, None]
            scales.append(sc)
        return {"values": values, "scale": torch.stack(scales, 1), "zero": torch.stack(zeros, 1).to(torch.uint8) if zeros else None}
    if case["op"] == "matvec":
        K, g = case["K"], case["group"]
        x = s["x"].double()
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=x.device)
        for j in range(s["s"].shape[1]):  # one group at a time: sum x * code, less zero * sum x, times the scale
            k0, k1 = j * g, min(K, (j + 1) * g)
            q = s["q"][:, k0 // 2:(k1 + 1) // 2]
            even, odd = x[:, k0:k1:2], x[:, k0 + 1:k1:2]
            z = s["z"][:, j].double() if s["z"] is not None else 8.0
            part = even @ (q & 15).double().t() + odd @ (q >> 4)[:, :odd.shape[1]].double().t()
            y += (part - x[:, k0:k1].sum(1, keepdim=True) * z) * s["s"][:, j].double()
        return {"y": y if s["b"] is None else y + s["b"].double()}
    if case["op"] == "lookup":
        out = torch.empty(case["T"], case["D"], dtype=torch.float64, device=DEVICE)
        t = s["tokens"]
        if case["table"] == "int4":
            q = s["t"].index_select(0, t)
            out[:, 0::2], out[:, 1::2] = (q & 15).double() - 8, (q >> 4).double() - 8
        elif case["table"] == "e4m3":
            out.copy_(s["t"].index_select(0, t).view(torch.float8_e4m3fn).float())
        else:
            out.copy_(s["t"].index_select(0, t))
        if s["s"] is not None:
            size = case["group"] if case["table"] == "int4" else 128
            sc = s["s"].index_select(0, t).double()
            for j in range(sc.shape[1]):
                out[:, j * size:(j + 1) * size] *= sc[:, j:j + 1]
        return {"rows": out * s["alpha"]}
    # tokens in order; a row's sum is the difference of running sums at its ends
    t, g = s["tokens"], s["g"].double()
    keep = torch.ones_like(t, dtype=torch.bool) if s["pad_row"] is None else t != s["pad_row"]
    order = torch.argsort(t[keep], stable=True)
    t, g = t[keep][order], g[keep][order]
    d = torch.zeros(case["V"], case["D"], dtype=torch.float64, device=DEVICE)
    if t.numel():
        rows, counts = torch.unique_consecutive(t, return_counts=True)
        ends = counts.cumsum(0)
        c = F.pad(g.cumsum(0), (0, 0, 1, 0))
        d[rows] = (c[ends] - c[ends - counts]) * s["alpha"]
    return {"table": d}
