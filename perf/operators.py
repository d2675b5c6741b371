"""Cases of the few-token layer, the block-scaled product and the activation quantiser.

Each operator has a plain form here (elementary torch operations in 32 bits), the call a user makes
of the library, and its definition in 64 bits.  The inputs are drawn on the GPU from a seed.

  few       one mixture-of-experts layer forward for 1..16 tokens, bf16 or e4m3 block-scaled weights
  product   out = A W^T with e4m3 operands, A scaled per 1x128 group, W per 128x128 block
  quantize  e4m3 codes and fp32 scales per 1x128 group, of x or of silu(g) * u
"""
import math

import torch

own = False

G = 128                     # values per scale group, and the side of a weight block
E4M3_MAX = 448.0


def listed():
    return [
        # the smallest layer of the test suite, a full batch of few tokens: latency alone counts
        dict(name="few_tiny", op="few", T=16, H=256, E=8, k=2, I=128, S=0, Is=0, fp8=False,
             bias="none", masked=0),
        # one user decoding: three of 48 wide experts and the shared one, 881 MB of weights
        dict(name="few_one", op="few", T=1, H=7168, E=48, k=3, I=5120, S=1, Is=5120, fp8=False,
             bias="none", masked=0),
        # a padded batch of many small experts with a skewed load: 11 of 16 rows are real
        dict(name="few_padded", op="few", T=16, H=7168, E=256, k=8, I=2048, S=1, Is=2048, fp8=False,
             bias="normal", masked=5),
        # one token of the e4m3 layer: 9 experts, 396 MB
        dict(name="few_fp8_one", op="few", T=1, H=7168, E=256, k=8, I=2048, S=1, Is=2048, fp8=True,
             bias="zipf", masked=0),
        # the e4m3 layer's ragged sizes: a shared expert of another width, 13 tokens, no power of two
        dict(name="few_fp8_odd", op="few", T=13, H=1920, E=40, k=5, I=640, S=1, Is=896, fp8=True,
             bias="zipf", masked=2),
        # a dense projection for one token: a stream of 29 MB of weights
        dict(name="product_one", op="product", M=1, N=4096, K=7168, fp32=False),
        # sizes that fill no tile: rows, features, and a last scale group of 48
        dict(name="product_odd", op="product", M=77, N=1111, K=1200, fp32=True),
        # a decode batch through a down projection
        dict(name="product_batch", op="product", M=256, N=7168, K=2048, fp32=False),
        # a prefill micro-batch through the gate/up projection of a shared expert
        dict(name="product_prefill", op="product", M=8192, N=4096, K=7168, fp32=False),
        # a decode batch's hidden states
        dict(name="quantize_batch", op="quantize", rows=128, cols=7168, gated=False, fp32=False,
             masked=0),
        # the hidden states of a prefill micro-batch
        dict(name="quantize_prefill", op="quantize", rows=8192, cols=7168, gated=False, fp32=False,
             masked=0),
        # gate and up outputs of an odd batch, some rows of it padding, a last group of 16
        dict(name="quantize_gated", op="quantize", rows=4099, cols=2064, gated=True, fp32=True,
             masked=900),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["few", "few", "product", "product", "quantize"])
    if op == "few":
        while True:
            T, k = rng.randint(1, 16), rng.randint(1, 8)
            c = dict(op="few", T=T, H=G * _log(rng, 1, 56), E=_log(rng, k, 256), k=k,
                     I=G * _log(rng, 1, 40), S=rng.randint(0, 1), Is=0, fp8=rng.random() < 0.5,
                     bias=rng.choice(["none", "normal", "zipf"]),
                     masked=rng.choice([0, 0, rng.randint(0, T - 1)]))
            if c["S"]:
                c["Is"] = G * _log(rng, 1, 40)
            # no more weights, and no more of them selected, than the largest listed layer
            if (c["E"] * c["I"] * c["H"] <= 256 * 2048 * 7168 and
                    (T * k * c["I"] + c["Is"]) * c["H"] <= 128 * 2048 * 7168):
                return c
    if op == "product":
        while True:
            c = dict(op="product", M=_log(rng, 1, 8192), N=_log(rng, 16, 10240),
                     K=16 * _log(rng, 2, 448), fp32=rng.random() < 0.3)
            if c["M"] * c["N"] * c["K"] <= 8192 * 4096 * 7168:
                return c
    rows = _log(rng, 1, 8192)
    return dict(op="quantize", rows=rows, cols=16 * _log(rng, 2, 448), gated=rng.random() < 0.5,
                fp32=rng.random() < 0.5, masked=rng.choice([0, rng.randint(0, rows - 1)]))


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, sigma=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)


def _quantize_weights(w):
    """bf16 [R, C] -> e4m3 [R, C] and fp32 scales of its 128x128 blocks, as a checkpoint holds them."""
    R, C = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -C % G, 0, -R % G))
    p = p.view(p.shape[0] // G, G, p.shape[1] // G, G)
    amax = p.abs().amax((1, 3))
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (p / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(-1, p.shape[2] * G)[:R, :C].contiguous().view(
        torch.float8_e4m3fn), s


def _fp8_weights(gen, groups, rows, cols, sigma):
    q = torch.empty(groups, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(groups, -(-rows // G), -(-cols // G), device="cuda")
    for g in range(groups):
        q[g], s[g] = _quantize_weights(_normal(gen, (rows, cols), sigma))
    return q, s


def _mask(gen, rows, masked):
    if not masked:
        return None
    valid = torch.ones(rows, dtype=torch.uint8, device="cuda")
    valid[torch.randperm(rows, generator=gen, device="cuda")[:masked]] = 0
    return valid


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "few":
        T, H, E, I, Is = c["T"], c["H"], c["E"], c["I"], c["Is"]
        st["x"] = _normal(gen, (T, H))
        st["valid"] = _mask(gen, T, c["masked"])
        w = {"router_w": _normal(gen, (E, H), 1 / math.sqrt(H), torch.float32), "router_b": None}
        if c["bias"] == "normal":
            w["router_b"] = _normal(gen, (E,), 1.0, torch.float32)
        elif c["bias"] == "zipf":
            rank = torch.randperm(E, generator=gen, device="cuda") + 1
            w["router_b"] = -1.1 * torch.log(rank.float())
        if c["fp8"]:
            w["w_gate_up"], w["s_gate_up"] = _fp8_weights(gen, E, 2 * I, H, 0.02)
            w["w_down"], w["s_down"] = _fp8_weights(gen, E, H, I, 0.02)
            if c["S"]:
                (w["ws_gate_up"],), (w["ss_gate_up"],) = _fp8_weights(gen, 1, 2 * Is, H, 0.02)
                (w["ws_down"],), (w["ss_down"],) = _fp8_weights(gen, 1, H, Is, 0.02)
        else:
            w["w_gate_up"] = _normal(gen, (E, 2 * I, H), 0.02)
            w["w_down"] = _normal(gen, (E, H, I), 0.02)
            if c["S"]:
                w["ws_gate_up"] = _normal(gen, (2 * Is, H), 0.02)
                w["ws_down"] = _normal(gen, (H, Is), 0.02)
        st["w"] = w
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        if own:
            import mixture_experts_fp32_b200 as moe
            st["plan"] = moe.Plan(max_tokens=T, hidden=H, num_experts=E, top_k_max=c["k"], inter=I,
                                  num_shared=c["S"], shared_inter=Is,
                                  wtype=moe.MOE_W_FP8_E4M3_B128 if c["fp8"] else moe.MOE_W_BF16)
            st["weights"] = st["plan"].weights(**w)
    elif c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        st["a"], st["sa"] = _plain_quantize(_normal(gen, (M, K)).float())
        (st["b"],), (st["sb"],) = _fp8_weights(gen, 1, N, K, 0.02)
        st["out"] = torch.empty(M, N, dtype=torch.float32 if c["fp32"] else torch.bfloat16,
                                device="cuda")
        if own:
            import mixture_experts_fp32_b200 as moe
            st["product"] = moe.Product(max_rows=M, n=N, k=K, out_dtype=st["out"].dtype)
    else:
        rows, cols = c["rows"], c["cols"]
        st["x"] = _normal(gen, (rows, cols * (2 if c["gated"] else 1)), 1.0,
                          torch.float32 if c["fp32"] else torch.bfloat16)
        st["valid"] = _mask(gen, rows, c["masked"])
        st["codes"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.empty(rows, -(-cols // G), device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _plain_quantize(v):
    """fp32 [..., K] -> e4m3 codes and the fp32 scale of each group of 128 along K."""
    K = v.shape[-1]
    p = torch.nn.functional.pad(v, (0, -K % G)).unflatten(-1, (-1, G))
    amax = p.abs().amax(-1)
    # divided by a tensor: torch multiplies by the reciprocal of a number, another rounding
    s = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    q = (p / s[..., None]).flatten(-2)[..., :K].contiguous()
    return q.to(torch.float8_e4m3fn), s


def _spread(s, K):
    return s.repeat_interleave(G, -1)[..., :K]


def _rounded(v):
    """What the e4m3 codes and scales of v stand for."""
    q, s = _plain_quantize(v)
    return q.float() * _spread(s, v.shape[-1])


def _blocks(q, s):
    """What e4m3 weights [..., R, C] with 128x128 block scales stand for."""
    R, C = q.shape[-2:]
    return q.float() * _spread(s, C).repeat_interleave(G, -2)[..., :R, :]


def _plain_mlp(x, gate_up, down, act):
    """x [P, H] through each row's own gate/up [P, 2I, H] and down [P, H, I] weights."""
    gu = torch.bmm(gate_up, act(x)[:, :, None])[:, :, 0]
    g, u = gu.chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    return torch.bmm(down, act(h)[:, :, None])[:, :, 0]


def _plain_few(c, w, x, valid):
    T, H, k = c["T"], c["H"], c["k"]
    x = x.float()
    if valid is not None:
        x = torch.where(valid[:, None] != 0, x, torch.zeros_like(x))
    logits = x @ w["router_w"].t()
    if w["router_b"] is not None:
        logits = logits + w["router_b"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].reshape(-1)
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    act = _rounded if c["fp8"] else (lambda v: v)
    if c["fp8"]:
        gate_up, down = _blocks(w["w_gate_up"].view(torch.uint8)[ids].view(torch.float8_e4m3fn),
                                w["s_gate_up"][ids]), _blocks(
            w["w_down"].view(torch.uint8)[ids].view(torch.float8_e4m3fn), w["s_down"][ids])
    else:
        gate_up, down = w["w_gate_up"][ids].float(), w["w_down"][ids].float()
    y = _plain_mlp(x.repeat_interleave(k, 0), gate_up, down, act).view(T, k, H)
    out = (p[:, :, None] * y).sum(1)
    if c["S"]:
        if c["fp8"]:
            gu, dn = _blocks(w["ws_gate_up"], w["ss_gate_up"]), _blocks(w["ws_down"], w["ss_down"])
        else:
            gu, dn = w["ws_gate_up"].float(), w["ws_down"].float()
        g, u = (act(x) @ gu.t()).chunk(2, 1)
        out = out + act(g / (1 + torch.exp(-g)) * u) @ dn.t()
    if valid is not None:
        out = torch.where(valid[:, None] != 0, out, torch.zeros_like(out))
    return out.to(torch.bfloat16)


def run(st):
    c = st["case"]
    if c["op"] == "few":
        if own:
            st["plan"].forward_few(st["weights"], st["x"], st["valid"], c["k"], st["out"])
            return st["out"]
        return _plain_few(c, st["w"], st["x"], st["valid"])
    if c["op"] == "product":
        if own:
            st["product"].forward(st["a"], st["sa"], st["b"], st["sb"], st["out"])
            return st["out"]
        a = st["a"].float() * _spread(st["sa"], c["K"])
        return (a @ _blocks(st["b"], st["sb"]).t()).to(st["out"].dtype)
    if own:
        import mixture_experts_fp32_b200 as moe
        moe.moe_quantize_groups(st["x"], st["codes"], st["scales"], valid=st["valid"],
                                gated=c["gated"])
        return {"codes": st["codes"], "scales": st["scales"]}
    v = st["x"].float()
    if c["gated"]:
        g, u = v.chunk(2, 1)
        v = g / (1 + torch.exp(-g)) * u
    if st["valid"] is not None:
        v = torch.where(st["valid"][:, None] != 0, v, torch.zeros_like(v))
    codes, scales = _plain_quantize(v)
    return {"codes": codes, "scales": scales}


def work(case):
    c = case
    if c["op"] == "few":
        T, H, E, k, b = c["T"] - c["masked"], c["H"], c["E"], c["k"], 1 if c["fp8"] else 2
        # distinct experts that T tokens select, were every expert as likely as the next
        active = E * (1 - (1 - k / E) ** T)
        shared = c["S"] * c["Is"] if T else 0
        weights = 3 * H * (active * c["I"] + shared) * b
        return {"bytes": weights + 4 * E * H * (T > 0) + 2 * T * H + 2 * c["T"] * H,
                "flops": 2 * T * H * (3 * (k * c["I"] + shared) + E)}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // G)
        return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // G)) + M * N * (4 if c["fp32"] else 2),
                "flops": 2 * M * N * K}
    rows, cols = c["rows"], c["cols"]
    size = (4 if c["fp32"] else 2) * (2 if c["gated"] else 1)
    return {"bytes": (rows - c["masked"]) * cols * size + rows * (cols + 4 * -(-cols // G)),
            "flops": (rows - c["masked"]) * cols * (8 if c["gated"] else 3)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_e4m3(v):
    """The e4m3 value nearest each v (ties to even, |v| <= 448): 3 bits of fraction, the least
    normal exponent -6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_groups(v):
    """(code values, scales) of float64 [R, K].  The format rounds three times: the scale to the 32
    bits it is stored in, v / scale to 32 bits (hidden states in bf16 often fall on the border of two
    codes, which the unrounded scale would decide otherwise), and that to e4m3."""
    codes, scales = torch.empty_like(v), []
    for k0 in range(0, v.shape[1], G):
        part = v[:, k0:k0 + G]
        s = (part.abs().amax(1) / E4M3_MAX).float().double()
        s[s == 0] = 1.0
        codes[:, k0:k0 + G] = _exact_e4m3((part / s[:, None]).float().double())
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _exact_matrix(q, s=None):
    m = q.double()
    if s is not None:
        for i, row in enumerate(s.double().repeat_interleave(G, 1)[:, :m.shape[1]]):
            m[i * G:i * G + G] *= row
    return m


def _exact_values(v, fp8):
    if not fp8:
        return v
    codes, scales = _exact_groups(v)
    for g in range(scales.shape[1]):
        codes[:, g * G:g * G + G] *= scales[:, g:g + 1]
    return codes


def _exact_expert(x, gu, sgu, dn, sdn, fp8):
    z = _exact_values(x, fp8) @ _exact_matrix(gu, sgu).t()
    half = z.shape[1] // 2
    h = torch.nn.functional.silu(z[:, :half]) * z[:, half:]
    return _exact_values(h, fp8) @ _exact_matrix(dn, sdn).t()


def exact(case, seed):
    c = case
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "product":
        a = st["a"].double()
        for g in range(st["sa"].shape[1]):
            a[:, g * G:g * G + G] *= st["sa"][:, g:g + 1].double()
        return a @ _exact_matrix(st["b"], st["sb"]).t()
    if c["op"] == "quantize":
        v = st["x"].double()
        if c["gated"]:
            v = torch.nn.functional.silu(v[:, :c["cols"]]) * v[:, c["cols"]:]
        if st["valid"] is not None:
            v[st["valid"] == 0] = 0.0
        codes, scales = _exact_groups(v)
        return {"codes": codes, "scales": scales}
    w, fp8 = st["w"], c["fp8"]
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    real = [t for t in range(c["T"]) if st["valid"] is None or int(st["valid"][t])]
    if not real:
        return out
    x = st["x"][real].double()
    logits = x @ w["router_w"].double().t()
    if w["router_b"] is not None:
        logits += w["router_b"].double()
    picked = {}                                     # expert -> [(row of x, weight)]
    for r, row in enumerate(logits.tolist()):
        best = sorted(range(c["E"]), key=lambda e: (-row[e], e))[:c["k"]]
        p = [math.exp(row[e] - row[best[0]]) for e in best]
        for e, v in zip(best, p):
            picked.setdefault(e, []).append((r, v / sum(p)))
    for e, rows in picked.items():
        r = [i for i, _ in rows]
        y = _exact_expert(x[r], w["w_gate_up"][e], w["s_gate_up"][e] if fp8 else None,
                          w["w_down"][e], w["s_down"][e] if fp8 else None, fp8)
        weight = torch.tensor([p for _, p in rows], dtype=torch.float64, device="cuda")
        out[torch.tensor(real, device="cuda")[r]] += weight[:, None] * y
    if c["S"]:
        out[real] += _exact_expert(x, w["ws_gate_up"], w.get("ss_gate_up"), w["ws_down"],
                                   w.get("ss_down"), fp8)
    return out
