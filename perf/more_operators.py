"""RMS norm with the residual's addition, MXFP8 quantisation and the experts' grouped products as measured cases.

Each case is one pass through one operator in two forms: the plain form in elementary torch operations (`own` false) and
the framework's own call (`own` true). `exact` gives the same outputs from the definitions in 64 bits.

Definitions:
  norm      h = x + residual, rounded to their type (h = x without a residual); r = 1 / sqrt(mean(h^2) + eps) of a row;
            y = h r g, in the type of x or in MXFP8. Backward, from dy and the gradient dh that reaches h from elsewhere:
            dx = dh + r (g dy - h r^2 mean(g dy h)), which is the residual's gradient too; dg = sum over rows of dy h r.
  mxfp8     blocks of 32 along the last axis: e = ceil(log2(amax / 448)), at least -127; scale byte e + 127; elements are
            E4M3, x / 2^e rounded to nearest, ties to even.
  grouped   rows [offsets[e], offsets[e + 1]) belong to expert e: y_r = W_e x_r, dx_r = W_e^T dy_r,
            dW_e = sum over its rows of dy_r x_r^T. Rows outside every group give zeros, groups without rows dW_e = 0.
  grouped8  the first of these with both operands MXFP8.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # one decode step of 16 streams: the norm in front of 8-bit experts, latency counts
        dict(name="norm_decode_t16", op="norm", rows=16, hidden=1024, dtype="bf16", residual=True, form="mxfp8"),
        # an odd prompt in half precision, in front of the router
        dict(name="norm_prompt_t2047", op="norm", rows=2047, hidden=2560, dtype="f16", residual=True, form="plain"),
        # a training step without a residual over rows of an odd width
        dict(name="norm_train_t1111x1001", op="norm", rows=1111, hidden=1001, dtype="f32", residual=False, form="train"),
        # a training step over many tokens: forward, and all gradients
        dict(name="norm_train_t16384x4096", op="norm", rows=16384, hidden=4096, dtype="bf16", residual=True,
             form="train"),
        # the activations of a prompt: quantised and read back
        dict(name="quantize_prompt_2047x2560", op="quantize", rows=2047, cols=2560, dtype="bf16"),
        # a layer's expert weights quantised once at load
        dict(name="quantize_weights_65536x1024", op="quantize", rows=65536, cols=1024, dtype="f32"),
        # one decode step of 16 streams through the experts' first product: bound by the touched experts' bytes
        dict(name="grouped_decode_t16", op="grouped", tokens=16, top_k=8, experts=96, k=1024, n=1024, dtype="bf16",
             routing="uniform", masked=0.0, train=False),
        # a short odd prompt through many narrow experts, some tokens masked, half precision
        dict(name="grouped_prompt_t111", op="grouped", tokens=111, top_k=10, experts=128, k=2560, n=640, dtype="f16",
             routing="zipf", masked=0.1, train=False),
        # a training micro-batch with uneven popularity: the product and both gradients
        dict(name="grouped_train_t2048", op="grouped", tokens=2048, top_k=8, experts=96, k=1024, n=1024, dtype="bf16",
             routing="zipf", masked=0.0, train=True),
        # a training step through few wide experts: bound by the matrix cores
        dict(name="grouped_train_t8192_wide", op="grouped", tokens=8192, top_k=2, experts=8, k=2048, n=4096,
             dtype="bf16", routing="uniform", masked=0.0, train=True),
        # one decode step with 8-bit operands
        dict(name="grouped8_decode_t16", op="grouped8", tokens=16, top_k=8, experts=96, k=1024, n=1024,
             routing="uniform", masked=0.0),
        # a prompt with 8-bit operands, uneven popularity
        dict(name="grouped8_prefill_t2048", op="grouped8", tokens=2048, top_k=8, experts=96, k=1024, n=1024,
             routing="zipf", masked=0.0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "grouped", "grouped", "grouped8"])
    if op == "norm":
        form = rng.choice(["plain", "train", "mxfp8"])
        hidden = 32 * _spread(rng, 2, 256) if form == "mxfp8" else _spread(rng, 64, 8192)
        return dict(op=op, rows=_spread(rng, 1, min(16384, 16384 * 4096 // hidden)), hidden=hidden,
                    dtype=rng.choice(["f32", "bf16", "f16"] if hidden <= 2048 else ["bf16", "f16"]),
                    residual=rng.random() < 0.7, form=form)
    if op == "quantize":
        cols = 32 * _spread(rng, 1, 256)
        return dict(op=op, rows=_spread(rng, 1, min(65536, 65536 * 1024 // cols)), cols=cols,
                    dtype=rng.choice(["f32", "bf16", "f16"]))
    experts = _spread(rng, 2, 128)
    top_k = min(experts, _spread(rng, 1, 10))
    if op == "grouped":
        k, n = 8 * _spread(rng, 16, 320), 8 * _spread(rng, 16, 320)
        case = dict(dtype=rng.choice(["bf16", "f16"]), train=rng.random() < 0.6)
    else:
        k, n = 32 * _spread(rng, 4, 80), 8 * _spread(rng, 16, 320)
        case = dict()
    tokens = _spread(rng, 1, max(1, min(4096, 16384 * 2048 * 4096 // (top_k * k * n))))
    return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, k=k, n=n, routing=rng.choice(["uniform", "zipf"]),
                masked=rng.choice([0.0, 0.1]), **case)


# ---------------------------------------------------------------- plain forms

def _scale_exponent(amax):
    """ceil(log2(amax / 448)), at least -127: amax = m * 2^x with m in [0.5, 1), and 448 = 0.875 * 2^9."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875).to(x.dtype), torch.full_like(x, -127)).clamp(min=-127)


def _power(e):
    """2^e as fp32 for whole e of [-127, 127], from its bits (2^-127 is a subnormal number)."""
    e = e.to(torch.int32)
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _codes_of(x):
    """fp32 [..., K] -> (E4M3 bytes uint8 [..., K], scale bytes uint8 [..., K / 32])."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    e = _scale_exponent(b.abs().amax(-1))
    v = b * _power(-e).unsqueeze(-1)
    return v.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), (e + 127).to(torch.uint8)


def _values_of(codes, scales):
    """fp32 values of E4M3 bytes [..., K] and scale bytes [..., K / 32]."""
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).reshape(*codes.shape[:-1], -1, 32)
    return (v * _power(scales.to(torch.int32) - 127).unsqueeze(-1)).reshape(codes.shape)


def _norm(state):
    x, g = state["x"], state["weight"].to(torch.float32)
    h = x if state["residual"] is None else (x.to(torch.float32) + state["residual"].to(torch.float32)).to(x.dtype)
    v = h.to(torch.float32)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    y = v * r * g
    if state["form"] == "mxfp8":
        out = dict(values=_values_of(*_codes_of(y)).to(torch.bfloat16))
    else:
        out = dict(y=y.to(x.dtype))
    if state["residual"] is not None:
        out["h"] = h
    if state["form"] == "train":
        dy = state["dy"].to(torch.float32)
        t = dy * g
        d = r * (t - v * (r * r * (t * v).mean(-1, keepdim=True)))
        if state["dh"] is not None:
            d = d + state["dh"].to(torch.float32)
        out.update(dx=d.to(x.dtype), dweight=(dy * v * r).sum(0).to(state["weight"].dtype))
    return out


def _places(state):
    """Where each row stands in a block of `cap` rows an expert (one more row for those outside every group)."""
    off, rows, cap, E = state["offsets"].to(torch.int64), state["rows"], state["cap"], state["experts"]
    r = torch.arange(rows, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    there = (r >= off[0]) & (e < E)
    e = e.clamp(max=E - 1)
    return torch.where(there, e * cap + r - off[e], torch.full_like(r, E * cap)), there.unsqueeze(-1)


def _padded(state, at, rows):
    a = torch.zeros(state["experts"] * state["cap"] + 1, rows.shape[1], dtype=torch.float32, device=rows.device)
    a[at] = rows.to(torch.float32)
    return a[:-1].reshape(state["experts"], state["cap"], -1)


def _gathered(state, at, there, blocks):
    flat = blocks.reshape(state["experts"] * state["cap"], -1)
    return torch.where(there, flat[at.clamp(max=flat.shape[0] - 1)], torch.zeros((), device=flat.device))


def _grouped(state):
    at, there = _places(state)
    x, w, dtype = state["x"], state["w"].to(torch.float32), state["x"].dtype
    a = _padded(state, at, x)
    out = dict(y=_gathered(state, at, there, torch.bmm(a, w.transpose(1, 2).contiguous())).to(dtype))
    if state["train"]:
        d = _padded(state, at, state["dy"])
        out["dx"] = _gathered(state, at, there, torch.bmm(d, w)).to(dtype)
        out["dw"] = torch.bmm(d.transpose(1, 2).contiguous(), a).to(dtype)
    return out


def _grouped8(state):
    at, there = _places(state)
    a = _padded(state, at, _values_of(state["xq"], state["xs"]))
    w = _values_of(state["wq"], state["ws"]).transpose(1, 2).contiguous()
    return _gathered(state, at, there, torch.bmm(a, w)).to(torch.bfloat16)


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _outliers(g, x):
    """One value in a hundred twenty times as large, as activations have them."""
    return torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.01, x * 20.0, x)


def _groups(g, case):
    """Offsets of the routes of a batch, sorted by expert; the routes of masked tokens stand in front of them."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    score = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    if case["routing"] == "zipf":
        rank = torch.randperm(E, generator=g, device="cuda").to(torch.float32) + 1.0
        score = score - 1.1 * torch.log(rank)
    ids = torch.sort(score, dim=1, descending=True)[1][:, :k]
    if case["masked"]:
        ids = ids.masked_fill((torch.rand(T, generator=g, device="cuda") < case["masked"]).unsqueeze(-1), -1)
    counts = torch.bincount(ids.reshape(-1) + 1, minlength=E + 1)
    return torch.cumsum(counts, 0).to(torch.int32), max(1, int(counts[1:].max()))


def _inputs(case, seed):
    g, op = _generator(seed), case["op"]
    if op == "norm":
        T, H, dtype = case["rows"], case["hidden"], DTYPES[case["dtype"]]
        s = dict(op=op, form=case["form"], x=_normal(g, T, H).to(dtype), residual=None, dy=None, dh=None,
                 weight=(1.0 + 0.2 * _normal(g, H)).to(dtype))
        if case["residual"]:
            s["residual"] = _outliers(g, _normal(g, T, H)).to(dtype)
        if case["form"] == "train":
            s["dy"] = _normal(g, T, H).to(dtype)
            if case["residual"]:
                s["dh"] = _normal(g, T, H).to(dtype)
        return s
    if op == "quantize":
        return dict(op=op, x=_outliers(g, _normal(g, case["rows"], case["cols"])).to(DTYPES[case["dtype"]]))
    E, K, N = case["experts"], case["k"], case["n"]
    rows = case["tokens"] * case["top_k"]
    offsets, cap = _groups(g, case)
    s = dict(op=op, offsets=offsets, cap=cap, experts=E, rows=rows)
    if op == "grouped8":
        s["xq"], s["xs"] = _codes_of(_normal(g, rows, K))
        s["wq"], s["ws"] = _codes_of(_normal(g, E, N, K) / math.sqrt(K))
        return s
    dtype = DTYPES[case["dtype"]]
    s.update(train=case["train"], x=_normal(g, rows, K).to(dtype), w=(_normal(g, E, N, K) / math.sqrt(K)).to(dtype))
    if case["train"]:
        s["dy"] = _normal(g, rows, N).to(dtype)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _plain(state):
    op = state["op"]
    if op == "norm":
        return _norm(state)
    if op == "quantize":
        codes, scales = _codes_of(state["x"].to(torch.float32))
        return dict(values=_values_of(codes, scales).to(state["x"].dtype), scales=scales)
    return _grouped(state) if op == "grouped" else _grouped8(state)


def _own(state):
    from trellis_quantized_moe_tmoe_amd import grouped, mxfp8, norm
    op = state["op"]
    if op == "norm":
        if state["form"] == "mxfp8":
            codes, scales, h = norm.rms_norm_mxfp8(state["x"], state["weight"], residual=state["residual"], eps=EPS)
            out = dict(values=mxfp8.dequantize(codes, scales, torch.bfloat16))
        else:
            y, h, rstd = norm.rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS)
            out = dict(y=y)
        if state["residual"] is not None:
            out["h"] = h
        if state["form"] == "train":
            out["dx"], out["dweight"] = norm.backward(h, state["weight"], rstd, state["dy"], dh=state["dh"])
        return out
    if op == "quantize":
        codes, scales = mxfp8.quantize(state["x"])
        return dict(values=mxfp8.dequantize(codes, scales, state["x"].dtype), scales=scales)
    if op == "grouped8":
        return mxfp8.grouped_linear(state["xq"], state["xs"], state["wq"], state["ws"], state["offsets"],
                                    out_dtype=torch.bfloat16)
    out = dict(y=grouped.linear(state["x"], state["w"], state["offsets"]))
    if state["train"]:
        out["dx"] = grouped.grad_x(state["dy"], state["w"], state["offsets"])
        out["dw"] = grouped.grad_w(state["dy"], state["x"], state["offsets"])
    return out


# ---------------------------------------------------------------- 64 bits

def _exact_rounded(x):
    """Values of the MXFP8 rounding of float64 x [rows][cols], and its scale bytes, from the spacing of E4M3."""
    b = x.reshape(-1, 32)
    amax = b.abs().max(1).values
    e = torch.full_like(amax, -127.0)
    some = amax > 0
    e[some] = torch.ceil(torch.log2(amax[some] / 448.0))
    e = torch.where(some & (amax <= 448.0 * torch.exp2(e - 1)), e - 1, e)        # log2's own rounding
    e = torch.where(some & (amax > 448.0 * torch.exp2(e)), e + 1, e).clamp(min=-127.0)
    m = b / torch.exp2(e)[:, None]
    binade = torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6)))
    binade = torch.where(torch.exp2(binade) > m.abs().clamp(min=2.0 ** -6), binade - 1, binade)
    step = torch.exp2(binade - 3)                                                # three bits behind the leading one
    v = torch.round(m / step) * step * torch.exp2(e)[:, None]                    # ties to even
    return v.reshape(x.shape), (e + 127).to(torch.uint8).reshape(*x.shape[:-1], -1)


def _exact_values(codes, scales):
    c = codes.to(torch.int64)
    ex, man = (c >> 3) & 15, (c & 7).double()
    v = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex.double() - 7))
    v = torch.where(c >= 128, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "norm":
        x, g, n = s["x"], s["weight"].double(), case["hidden"]
        h = x if s["residual"] is None else (x.double() + s["residual"].double()).to(x.dtype)
        v = h.double()
        root = torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / n + EPS)
        unit = v / root
        out = dict(values=_exact_rounded(unit * g)[0]) if case["form"] == "mxfp8" else dict(y=unit * g)
        if s["residual"] is not None:
            out["h"] = x.double() + s["residual"].double()
        if case["form"] == "train":
            dy = s["dy"].double()
            along = torch.sum(dy * g * unit, 1, keepdim=True) / n
            out["dx"] = (dy * g - unit * along) / root
            if s["dh"] is not None:
                out["dx"] = out["dx"] + s["dh"].double()
            out["dweight"] = torch.sum(dy * unit, 0)
        return out
    if op == "quantize":
        return dict(values=_exact_rounded(s["x"].double())[0], scales=None)
    off = s["offsets"].tolist()
    if op == "grouped8":
        x, y = _exact_values(s["xq"], s["xs"]), torch.zeros(s["rows"], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            a, b = off[e], off[e + 1]
            if b > a:
                y[a:b] = torch.matmul(x[a:b], _exact_values(s["wq"][e], s["ws"][e]).t().contiguous())
        return y
    out = dict(y=torch.zeros(s["rows"], case["n"], dtype=torch.float64, device="cuda"))
    if case["train"]:
        out["dx"] = torch.zeros(s["rows"], case["k"], dtype=torch.float64, device="cuda")
        out["dw"] = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if b == a:
            continue
        x, w = s["x"][a:b].double(), s["w"][e].double()
        out["y"][a:b] = torch.matmul(x, w.t().contiguous())
        if case["train"]:
            dy = s["dy"][a:b].double()
            out["dx"][a:b] = torch.matmul(dy, w)
            out["dw"][e] = torch.matmul(dy.t().contiguous(), x)
    return out


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "norm":
        n, s = case["rows"] * case["hidden"], size[case["dtype"]]
        res, train, out = 2 if case["residual"] else 0, case["form"] == "train", s
        if case["form"] == "mxfp8":              # written as codes and scales, read back, written as values
            out = 2 * 33 / 32 + 2
        back = (3 * s + (s if case["residual"] else 0)) if train else 0
        return dict(bytes=n * (s + res * s + out + back), flops=n * (16 if train else 6))
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (2 * size[case["dtype"]] + 2 * 33 / 32), flops=4 * n)
    R, K, N, E, k = case["tokens"] * case["top_k"], case["k"], case["n"], case["experts"], case["top_k"]
    touched = E * (1 - (1 - k / E) ** case["tokens"]) if k < E else E
    if op == "grouped8":
        return dict(bytes=(R + touched * N) * K * 33 / 32 + 2 * R * N, flops=2 * R * K * N)
    y, w, passes = 2 * R * (K + N), 2 * touched * N * K, 3 if case["train"] else 1
    dw = 2 * E * N * K if case["train"] else 0
    return dict(bytes=passes * y + (2 * w if case["train"] else w) + dw, flops=2 * passes * R * K * N)
