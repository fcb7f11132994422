"""What the framework's language-model operators are measured on.

Two groups: the 8-bit forward of a jointly sparsified and quantized linear
layer (tokens quantized to 8 bits with a scale each, optionally behind the
MLP's gate, and the integer product with a scale per token and per output
channel), and causal attention over packed prompts with grouped heads.

Each case is one pass as a user's program makes it. `own` false: elementary
torch operations in 32 bits, rounded once at the end; `own` true: the
framework's entry points.
"""

import math

import torch

own = False



# ------------------------------------------------------------------- cases

def _lin(name, n, d_in, d_out, out):
    return {"name": name, "op": "linear", "n": n, "d_in": d_in, "d_out": d_out, "out": out}


def _gated(name, n, d_in, d_out):
    return {"name": name, "op": "gated", "n": n, "d_in": d_in, "d_out": d_out, "out": "bf16"}


def _attn(name, lens, heads, kv_heads, width):
    return {"name": name, "op": "attention", "lens": ",".join(map(str, lens)), "heads": heads, "kv_heads": kv_heads,
            "width": width}


def listed():
    return [
        # one generated token through the 5120-wide layer's query projection: launch and weight-read latency
        _lin("linear_one_token", 1, 5120, 8192, "bf16"),
        # a decoding batch through the widest reduction (down projection of the 25600-wide MLP)
        _lin("linear_batch16_wide", 16, 25600, 5120, "bf16"),
        # a short ragged prompt through the 768-wide layer, results in fp32
        _lin("linear_ragged_768", 333, 768, 768, "fp32"),
        # one calibration sequence, odd length, 11008-wide down projection, fp32 as the solver's other products give
        _lin("linear_down_11008", 2047, 11008, 4096, "fp32"),
        # two calibration sequences through gate/up
        _lin("linear_gate_4096_tokens", 4096, 5120, 25600, "bf16"),
        # a large calibration chunk through gate/up: the largest case
        _lin("linear_gate_16384_tokens", 16384, 5120, 25600, "bf16"),
        # the gated input of the down projection, a few decoded tokens
        _gated("gated_down_8_tokens", 8, 25600, 5120),
        # the same over two sequences and three odd tokens
        _gated("gated_down_4099_tokens", 4099, 25600, 5120),
        # a batch of very short prompts, 12 heads of width 64
        _attn("attention_short_prompts", [1, 7, 64, 128, 129, 300], 12, 12, 64),
        # calibration: eight sequences of 2048, 64 query heads on 8 key/value heads
        _attn("attention_calibration", [2048] * 8, 64, 8, 128),
        # packed prompts of very different lengths, no head sharing
        _attn("attention_packed_ragged", [5, 1777, 260, 2900, 33, 1024, 611, 97], 32, 32, 128),
        # one long prompt, one key/value head's group
        _attn("attention_long_prompt", [16384], 8, 1, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "attention", "attention"])
    if op == "attention":
        while True:
            width = rng.choice([64, 128])
            kv = rng.choice([1, 2, 4, 8, 12])
            heads = kv * rng.choice([1, 1, 2, 3, 4, 8])
            count = _log_int(rng, 1, 24)
            longest = _log_int(rng, 1, 16384)
            lens = [max(1, min(longest, _log_int(rng, 1, 16384))) for _ in range(count)]
            lens[rng.randrange(count)] = longest
            padded = count * heads * max(lens) ** 2
            if heads <= 64 and padded <= 8 * 16384 ** 2 and sum(lens) * heads <= 16384 * 64:
                c = _attn("", lens, heads, kv, width)
                break
    else:
        while True:
            n = _log_int(rng, 1, 16384)
            d_in = 32 * _log_int(rng, 8, 800)
            d_out = _log_int(rng, 64, 25600)
            if n * d_in * d_out <= 4e11 and n * d_in <= 12e7 and n * d_out <= 4e8:
                break
        c = _gated("", n, d_in, d_out) if op == "gated" else _lin("", n, d_in, d_out, rng.choice(["bf16", "bf16", "fp32"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, n, d):
    """Rows whose channels have very uneven scales, a hundredth of them outliers, as decoder layers' inputs do."""
    s = torch.exp(torch.randn(d, device="cuda", generator=g))
    s = torch.where(torch.rand(d, device="cuda", generator=g) < 0.01, 20 * s, s)
    x = torch.empty(n, d, device="cuda", dtype=torch.bfloat16)
    step = max(1, (1 << 27) // d)
    for a in range(0, n, step):
        b = min(n, a + step)
        x[a:b] = torch.randn(b - a, d, device="cuda", generator=g) * s
    return x


def _weights(g, d_out, d_in):
    """8-bit codes (less 128) and the row grid (scale, zero point) of a random layer: uniform and asymmetric, 256
    levels over the row's range, as the joint sparse and quantized sweep keeps them."""
    w = torch.randn(d_out, d_in, device="cuda", generator=g) / math.sqrt(d_in)
    lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
    scale = (hi - lo) / torch.full_like(hi, 255)
    zero = torch.round(-lo / scale)
    codes = (torch.round(w / scale[:, None]) + zero[:, None]).clamp(0, 255) - 128
    return codes.to(torch.int8), torch.stack([scale, zero], 1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    s = {"case": case, "info": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["op"] == "attention":
        lens = [int(v) for v in case["lens"].split(",")]
        t, h, kv, w = sum(lens), case["heads"], case["kv_heads"], case["width"]
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        # queries and keys whose scores have a standard deviation of two: neither flat nor one-hot
        s["Q"] = (math.sqrt(2) * torch.randn(t, h, w, device=dev, generator=g)).to(torch.bfloat16)
        s["K"] = (math.sqrt(2) * torch.randn(t, kv, w, device=dev, generator=g)).to(torch.bfloat16)
        s["V"] = torch.randn(t, kv, w, device=dev, generator=g).to(torch.bfloat16)
        s["O"] = torch.zeros(t, h, w, device=dev, dtype=torch.bfloat16)
        return s
    n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
    s["codes"], s["grid"] = _weights(g, d_out, d_in)
    if case["op"] == "gated":
        s["G"] = (1.5 * torch.randn(n, d_in, device=dev, generator=g)).to(torch.bfloat16)
        s["U"] = _activations(g, n, d_in)
    else:
        s["X"] = _activations(g, n, d_in)
    s["Xq"] = torch.empty(n, d_in, dtype=torch.int8, device=dev)
    s["scale"] = torch.empty(n, device=dev)
    s["sums"] = torch.empty(n, dtype=torch.int32, device=dev)
    s["Y"] = torch.empty(n, d_out, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=dev)
    return s


# --------------------------------------------------------------------- run

def _plain_linear(z, s):
    """y = s_t scale_r sum_k q_tk (c_rk - (zero_r - 128)), q = round(127 z / max|z|) of each row."""
    top = z.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(torch.div(127 * z, top)), torch.zeros_like(z))
    scale = torch.div(top, torch.full_like(top, 127))
    weights = s["codes"].float() - (s["grid"][:, 1:] - 128)
    return (torch.matmul(q, weights.t()) * scale * s["grid"][:, 0]).to(s["Y"].dtype)


def _plain_attention(s):
    lens, cu = s["lens"], s["cu"].long()
    most = max(lens)
    q, k, v = s["Q"], s["K"], s["V"]
    kv, w = k.shape[1], k.shape[2]
    group = q.shape[1] // kv
    at = cu[:-1, None] + torch.arange(most, device=q.device)               # [B, L] rows of the packed tensors
    there = at < cu[1:, None]
    at = at.clamp(max=q.shape[0] - 1)
    qp = q[at].float().unflatten(2, (kv, group)).permute(0, 2, 3, 1, 4)    # [B, kv, group, L, w]
    kp = k[at].float().permute(0, 2, 1, 3)[:, :, None]                     # [B, kv, 1, L, w]
    vp = torch.where(there[:, :, None, None], v[at].float(), 0.0).permute(0, 2, 1, 3)[:, :, None]
    x = torch.matmul(qp, kp.transpose(-1, -2)).mul_(1 / math.sqrt(w))
    i = torch.arange(most, device=q.device)
    x.masked_fill_(i[None, :] > i[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, vp) / total                                        # [B, kv, group, L, w]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                             # [B, L, heads, w]
    return o[there].to(q.dtype)                                            # row by row: the packed order


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import post_pruning_b200 as pp
        if op == "attention":
            pp.attention(s["Q"], s["K"], s["V"], s["cu"], s["O"], s["info"])
            return s["O"]
        if op == "gated":
            pp.quant_tokens_silu(s["G"], s["U"], s["Xq"], s["scale"], s["sums"], s["info"])
        else:
            pp.quant_tokens(s["X"], s["Xq"], s["scale"], s["sums"], s["info"])
        pp.linear_i8(s["Xq"], s["scale"], s["sums"], s["codes"], s["grid"], s["Y"], s["info"])
        return s["Y"]
    if op == "attention":
        return _plain_attention(s)
    if op == "gated":
        gate = s["G"].float()
        return _plain_linear(gate / (1 + torch.exp(-gate)) * s["U"].float(), s)
    return _plain_linear(s["X"].float(), s)


# -------------------------------------------------------------- what it needs

def work(case):
    if case["op"] == "attention":
        lens = [int(v) for v in case["lens"].split(",")]
        t, h, kv, w = sum(lens), case["heads"], case["kv_heads"], case["width"]
        return {"bytes": 2 * t * w * (2 * h + 2 * kv), "flops": 4 * w * h * sum(n * (n + 1) // 2 for n in lens)}
    n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
    reads = n * d_in * (4 if case["op"] == "gated" else 2) + d_out * d_in + 8 * d_out
    return {"bytes": reads + n * d_out * (2 if case["out"] == "bf16" else 4), "flops": 2 * n * d_in * d_out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        q, k, v = s["Q"], s["K"], s["V"]
        t, h, w = q.shape
        share = h // k.shape[1]
        o = torch.zeros(t, h, w, dtype=torch.float64, device=q.device)
        first = 0
        for n in s["lens"]:
            rows = slice(first, first + n)
            first += n
            lower = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
            for j in range(h):
                x = q[rows, j].double() @ k[rows, j // share].double().t() / w ** 0.5
                p = torch.softmax(x.masked_fill(~lower, -math.inf), dim=1)
                o[rows, j] = p @ v[rows, j // share].double()
        return o
    if case["op"] == "gated":
        x = torch.nn.functional.silu(s["G"].double()) * s["U"].double()
    else:
        x = s["X"].double()
    peak = x.abs().max(dim=1).values
    peak = torch.where(peak == 0, torch.ones_like(peak), peak)             # a row of zeros has codes of zero
    q = torch.round(x * 127 / peak[:, None])
    del x
    scale, zero = s["grid"].double().unbind(1)
    w = (s["codes"].double() + 128 - zero[:, None]) * scale[:, None]
    return (q * (peak[:, None] / 127)) @ w.t()
