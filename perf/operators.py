"""The serving operators around the quantized attention, as cases that can be timed and compared.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the calls a user makes:

* ``norm_rope``  RMS norm of every query and key head and its position rotation, in one pass
* ``append``     new tokens into the paged INT8 K / E4M3 V cache (norm and rotation in the same pass), and what was
                 written read back
* ``gather``     cached prefixes read back as 16-bit K and V
* ``decode``     attention of one new token per sequence over the paged cache
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
TINY_AMAX = 2.0 ** -100  # rows below it are stored as zeros


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's heads straight from the fused projection (strided), one token of each of 64 requests
        dict(name="norm_rope_step_t64", op="norm_rope", B=1, N=64, Hq=32, Hkv=8, d=128, rot=128, layout="packed",
             dtype="fp16", norm=True, weights="same", interleaved=False),
        # a video transformer's whole sequence, adjacent channels rotated as pairs
        dict(name="norm_rope_video_n32768", op="norm_rope", B=1, N=32768, Hq=24, Hkv=24, d=128, rot=128,
             layout="NHD", dtype="bf16", norm=True, weights="fp32", interleaved=True),
        # an odd length, a padded head size, only part of each head rotated
        dict(name="norm_rope_odd_d96", op="norm_rope", B=3, N=1537, Hq=16, Hkv=16, d=96, rot=48, layout="HND",
             dtype="fp16", norm=True, weights="same", interleaved=False),
        # a decode step's write: one token of each of 64 requests
        dict(name="append_step_b64", op="append", B=64, new=1, hist=2000, ragged=True, Hq=32, Hkv=8, d=128, rot=128,
             page=64, dtype="fp16", norm=True, interleaved=False, mean=False),
        # prompts of an LLM prefill batch
        dict(name="append_prompt_b4_n8192", op="append", B=4, new=8192, hist=0, ragged=False, Hq=32, Hkv=8, d=128,
             rot=128, page=64, dtype="fp16", norm=True, interleaved=False, mean=True),
        # ragged chunks behind cached prefixes; heads that were rotated before
        dict(name="append_chunk_d80", op="append", B=7, new=700, hist=900, ragged=True, Hq=8, Hkv=2, d=80, rot=0,
             page=16, dtype="bf16", norm=False, interleaved=False, mean=True),
        # one request's prefix
        dict(name="gather_b1_n1000", op="gather", B=1, max_len=1000, ragged=False, Hkv=8, d=128, page=64,
             dtype="fp16", mean=False),
        # the prefixes of a batch of chunked prompts
        dict(name="gather_b16_n8192", op="gather", B=16, max_len=8192, ragged=True, Hkv=8, d=128, page=64,
             dtype="bf16", mean=True),
        # one short request: latency
        dict(name="decode_b1_n500", op="decode", B=1, max_len=500, ragged=False, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16"),
        # the decode that follows the LLM prefill batch
        dict(name="decode_b4_n8192", op="decode", B=4, max_len=8192, ragged=False, Hq=32, Hkv=8, d=128, page=64,
             dtype="fp16"),
        # a loaded server: 64 requests of all lengths, padded slots among them
        dict(name="decode_b64_n16384", op="decode", B=64, max_len=16384, ragged=True, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16"),
        # one very long request
        dict(name="decode_b1_n131072", op="decode", B=1, max_len=131072, ragged=False, Hq=32, Hkv=8, d=128, page=256,
             dtype="fp16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "gather", "decode", "decode"])
    dtype = rng.choice(["fp16", "bf16"])
    d = rng.choice([40, 64, 80, 96, 128, 128, 160, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    rot = rng.choice([d, d, d // 2])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm_rope":
        B = rng.choice([1, 1, 2, 3])
        N = _log(rng, 1, min(32768, 150_000_000 // (B * (Hq + Hkv) * d)))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, rot=rot, dtype=dtype, norm=rng.random() < 0.8,
                    layout="packed" if B == 1 and rng.random() < 0.5 else rng.choice(["HND", "NHD"]),
                    weights=rng.choice(["none", "same", "fp32"]), interleaved=rng.random() < 0.4)
    if op == "append":
        B = _log(rng, 1, 96)
        new = _log(rng, 1, max(2, min(8192, 100_000_000 // (B * (Hq + 2 * Hkv) * d))))
        return dict(op=op, B=B, new=new, hist=_log(rng, 1, 1500), ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([0, rot]), page=page, dtype=dtype, norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.4, mean=rng.random() < 0.5)
    if op == "gather":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, max_len=_log(rng, 1, max(2, min(16384, 120_000_000 // (B * Hkv * d)))),
                    ragged=rng.random() < 0.7, Hkv=Hkv, d=d, page=page, dtype=dtype, mean=rng.random() < 0.5)
    B = _log(rng, 1, 96)
    return dict(op=op, B=B, max_len=_log(rng, 1, max(2, min(131072, 500_000_000 // (B * Hkv * d)))),
                ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)


def _lengths(n, most, ragged):
    """Lengths of a batch: all alike, or spread over 1..most, the first the longest and the last of four or more an empty slot."""
    if not ragged:
        return [most] * n
    out = [most] + [1 + int((most - 1) * (i * 0.6180339887498949 % 1.0)) for i in range(1, n)]
    if n >= 4:
        out[-1] = 0
    return out


def _append_lengths(case):
    """(new tokens, tokens before them) of every sequence."""
    new = _lengths(case["B"], case["new"], case["ragged"] and case["new"] > 1)
    hist = _lengths(case["B"], case["hist"], case["ragged"]) if case["hist"] else [0] * case["B"]
    return new, [h if n else 0 for n, h in zip(new, hist)]


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed, stream):
    return torch.Generator(device="cuda").manual_seed(seed * 64 + stream)


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _table(n, rot):
    """cos and sin of position x frequency, from angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _pages(lens, page, g):
    """A page table (-1 behind a sequence's pages) over pages handed out in random order, and how many there are."""
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(need)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _empty_cache(pages, Hkv, page, d):
    dc = -(-d // 16) * 16
    z = lambda *s, dtype: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    return dict(k8=z(pages, Hkv, page, dc, dtype=torch.int8), ks=z(pages, Hkv, page, dtype=torch.float32),
                v8=z(pages, Hkv, page, dc, dtype=torch.uint8), vs=z(pages, Hkv, page, dtype=torch.float32))


def _filled_cache(pages, Hkv, page, d, g):
    """Codes and scales as N(0, 1) keys and values leave them: the largest of d values at the end of the code range."""
    c = _empty_cache(pages, Hkv, page, d)
    top = math.sqrt(2 * math.log(2 * d))  # about the largest |x| of d
    step = max(1, 200_000_000 // (Hkv * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        c["k8"][i:i + n, :, :, :d] = (_normal((n, Hkv, page, d), g) * (127 / top)).round().clamp(-127, 127).to(torch.int8)
        c["v8"][i:i + n, :, :, :d] = (_normal((n, Hkv, page, d), g) * (448 / top)).clamp(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)
    c["ks"].copy_((0.1 * _normal(c["ks"].shape, g)).exp() * (top / 127))
    c["vs"].copy_((0.1 * _normal(c["vs"].shape, g)).exp() * (top / 448))
    return c


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _k_offset(Hkv, d, g):
    return _normal((Hkv, d), g) * 2


def prepare(case, seed):
    s, dt = dict(case), DTYPES[case["dtype"]]
    d, g = case["d"], _gen(seed, 0)
    if case["op"] == "norm_rope":
        B, N, Hq, Hkv = case["B"], case["N"], case["Hq"], case["Hkv"]
        if case["layout"] == "packed":  # views of the projection's rows [q heads | k heads | v heads]
            rows = _normal((N, Hq + 2 * Hkv, d), g, dt)
            s["q"], s["k"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
        elif case["layout"] == "NHD":
            s["q"], s["k"] = _normal((B, N, Hq, d), g, dt), _normal((B, N, Hkv, d), g, dt)
        else:
            s["q"], s["k"] = _normal((B, Hq, N, d), g, dt), _normal((B, Hkv, N, d), g, dt)
        n_pos = max(N, 4096)
        s["cos_sin"] = _table(n_pos, case["rot"])
        if case["layout"] == "packed":  # one token of each of N requests, at any position
            s["positions"] = torch.randint(0, n_pos, (N,), generator=g, device="cuda").to(torch.int32)
        else:
            s["positions"] = torch.arange(N, dtype=torch.int32, device="cuda")
        wt = {"none": None, "same": dt, "fp32": torch.float32}[case["weights"] if case["norm"] else "none"]
        s["q_weight"] = None if wt is None else (1 + 0.2 * _normal((d,), g)).to(wt)
        s["k_weight"] = None if wt is None else (1 + 0.2 * _normal((d,), g)).to(wt)
        return s
    if case["op"] == "append":
        new, hist = _append_lengths(case)
        lens = [n + h for n, h in zip(new, hist)]
        T, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
        rows = _normal((T, Hq + 2 * Hkv, d), g, dt)
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        s["k_mean"] = _k_offset(Hkv, d, g) if case["mean"] else None
        if case["mean"] and not case["norm"]:
            s["k"].add_(s["k_mean"])  # keys with a channel offset, which the mean removes
        s["page_table"], pages = _pages(lens, case["page"], g)
        s["cache"] = _empty_cache(pages, Hkv, case["page"], d)
        s["seq_lens"], s["starts"] = _ints(lens), _ints(hist)
        s["cu"] = _ints(_offsets(new))
        s["cos_sin"] = _table(max(lens), case["rot"]) if case["rot"] else None
        s["q_weight"] = (1 + 0.2 * _normal((d,), g)).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * _normal((d,), g)).to(dt) if case["norm"] else None
        s["T"] = T
        return s
    lens = _lengths(case["B"], case["max_len"], case["ragged"])
    s["page_table"], pages = _pages(lens, case["page"], g)
    s["cache"] = _filled_cache(pages, case["Hkv"], case["page"], d, g)
    if case["op"] == "gather":
        s["cu"], s["T"] = _ints(_offsets(lens)), sum(lens)
        s["k_mean"] = _k_offset(case["Hkv"], d, g) if case["mean"] else None
    else:
        s["seq_lens"] = _ints(lens)
        s["q"] = _normal((case["B"], case["Hq"], d), g, dt)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _norm_rope(x, w, s, cos_sin, positions):
    """x (..., heads, d) in 32 bits; positions of every index before the heads."""
    if s["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        if w is not None:
            x = x * w.float()
    if cos_sin is None:
        return x
    h = s["rot"] // 2
    row = cos_sin[positions.long()][..., None, :]
    cos, sin = row[..., :h], row[..., h:]
    y = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def _scale_and_inverse(x, top):
    amax = x.abs().amax(-1)
    keep = amax >= TINY_AMAX
    zero = torch.zeros_like(amax)
    return torch.where(keep, amax / top, zero), torch.where(keep, top / amax, zero)


def _places(s):
    """(page, slot) of every packed token, cu the packed offsets and `starts` each sequence's first position."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    pos = t - s["cu"][b]
    if s.get("starts") is not None:
        pos = pos + s["starts"][b]
    page = s["cache"]["ks"].shape[2]
    return s["page_table"][b, (pos // page).long()].long(), (pos % page).long(), pos


def _read(s):
    c, d = s["cache"], s["d"]
    page, slot, _ = _places(s)
    k = c["k8"][page, :, slot][..., :d].float() * c["ks"][page, :, slot][..., None]
    v = c["v8"].view(torch.float8_e4m3fn)[page, :, slot][..., :d].float() * c["vs"][page, :, slot][..., None]
    if s["k_mean"] is not None:
        k = k + s["k_mean"]
    return k.to(DTYPES[s["dtype"]]), v.to(DTYPES[s["dtype"]])


def _plain_append(s):
    c, d = s["cache"], s["d"]
    page, slot, pos = _places(s)
    q = _norm_rope(s["q"].float(), s["q_weight"], s, s["cos_sin"], pos)
    k = _norm_rope(s["k"].float(), s["k_weight"], s, s["cos_sin"], pos)
    if s["k_mean"] is not None:
        k = k - s["k_mean"]
    v = s["v"].float()
    ks, ki = _scale_and_inverse(k, 127.0)
    vs, vi = _scale_and_inverse(v, 448.0)
    code = torch.zeros((s["T"], s["Hkv"], c["k8"].shape[-1]), dtype=torch.int8, device="cuda")
    code[..., :d] = (k * ki[..., None]).round().clamp(-127, 127).to(torch.int8)
    c["k8"][page, :, slot] = code
    code = torch.zeros_like(code, dtype=torch.uint8)
    code[..., :d] = (v * vi[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    c["v8"][page, :, slot] = code
    c["ks"][page, :, slot] = ks
    c["vs"][page, :, slot] = vs
    k, v = _read(s)
    return dict(q=q.to(DTYPES[s["dtype"]]), k=k, v=v)


def _plain_decode(s):
    c, d, B, Hkv = s["cache"], s["d"], s["B"], s["Hkv"]
    page_size = c["ks"].shape[2]
    pos = torch.arange(s["max_len"], device="cuda")
    page, slot = s["page_table"][:, pos // page_size].long().clamp(min=0), (pos % page_size).expand(B, -1)
    seen = (pos < s["seq_lens"][:, None])[:, None, None]                                     # (B, 1, 1, L)
    k = c["k8"][page, :, slot][..., :d].float() * c["ks"][page, :, slot][..., None]          # (B, L, Hkv, d)
    q = s["q"].float().view(B, Hkv, -1, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(d))                      # (B, Hkv, G, L)
    del k
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    v = c["v8"].view(torch.float8_e4m3fn)[page, :, slot][..., :d].float() * c["vs"][page, :, slot][..., None]
    v = torch.where(seen.view(B, -1, 1, 1), v, 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    return out.view(B, -1, d).to(DTYPES[s["dtype"]])


def _plain(s):
    if s["op"] == "norm_rope":
        heads_last = s["layout"] != "HND"
        out = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.float() if heads_last else x.float().transpose(1, 2)
            y = _norm_rope(x, w, s, s["cos_sin"], s["positions"])
            out.append((y if heads_last else y.transpose(1, 2)).contiguous().to(DTYPES[s["dtype"]]))
        return dict(q=out[0], k=out[1])
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "gather":
        k, v = _read(s)
        return dict(k=k, v=v)
    return _plain_decode(s)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import quantized_attention_int8_b200 as qa
    if s["op"] == "norm_rope":
        q, k = qa.sage_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"],
                                    tensor_layout="HND" if s["layout"] == "HND" else "NHD", norm=s["norm"],
                                    interleaved=s["interleaved"])
        return dict(q=q, k=k)
    if s["op"] == "append":
        q = qa.sage_cache_append(s["cache"], s["k"], s["v"], s["page_table"], s["seq_lens"], s["cu"], q=s["q"],
                                 cos_sin=s["cos_sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 norm=s["norm"], interleaved=s["interleaved"], k_mean=s["k_mean"])
        k, v = qa.sage_cache_gather(s["cache"], s["page_table"], s["cu"], s["T"], s["d"], DTYPES[s["dtype"]],
                                    starts=s["starts"], k_mean=s["k_mean"])
        return dict(q=q, k=k, v=v)
    if s["op"] == "gather":
        k, v = qa.sage_cache_gather(s["cache"], s["page_table"], s["cu"], s["T"], s["d"], DTYPES[s["dtype"]],
                                    k_mean=s["k_mean"])
        return dict(k=k, v=v)
    return qa.sage_attn_decode(s["q"], s["cache"], s["page_table"], s["seq_lens"], s["max_len"])


# ------------------------------------------------------------------------------------------------ work
def work(case):
    d = case["d"]
    if case["op"] == "norm_rope":
        n, H = case["B"] * case["N"], case["Hq"] + case["Hkv"]
        rows = min(case["N"], max(case["N"], 4096))
        return dict(bytes=4.0 * n * H * d + 4.0 * rows * case["rot"] + 4.0 * case["N"],
                    flops=float(n * H * (4 * d * case["norm"] + 3 * case["rot"])))
    if case["op"] == "append":
        new, hist = _append_lengths(case)
        T, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
        tables = 4.0 * (sum(-(-(n + h) // case["page"]) - h // case["page"] for n, h in zip(new, hist)) + 3 * case["B"])
        rows = len({p for n, h in zip(new, hist) for p in range(h, h + n)})
        written = T * (2.0 * Hq * d + Hkv * (2 * d + 8))
        return dict(bytes=2.0 * T * (Hq + 2 * Hkv) * d + written + T * 4.0 * Hkv * d + tables + 4.0 * rows * case["rot"],
                    flops=float(T * ((Hq + Hkv) * (4 * d * case["norm"] + 3 * case["rot"]) + 8 * Hkv * d)))
    lens = _lengths(case["B"], case["max_len"], case["ragged"])
    total, Hkv = sum(lens), case["Hkv"]
    tables = 4.0 * (sum(-(-n // case["page"]) for n in lens) + case["B"])
    cached = total * Hkv * (2.0 * d + 8)
    if case["op"] == "gather":
        return dict(bytes=cached + tables + total * Hkv * 4.0 * d, flops=2.0 * total * Hkv * d)
    return dict(bytes=cached + tables + 4.0 * case["B"] * case["Hq"] * d, flops=4.0 * total * case["Hq"] * d)


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_rows(x, w, norm, cos, sin, interleaved):
    """RMS norm and rotation of rows x (tokens, heads, d); cos, sin (tokens, rot / 2)."""
    x = x.double()
    if norm:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()
        x = x if w is None else x * w.double()
    if cos is None:
        return x
    h = cos.shape[-1]
    turn = torch.complex(cos.double(), sin.double())[:, None]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., 2 * h:]], -1)
    z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
    return torch.cat([z.real, z.imag, x[..., 2 * h:]], -1)


def _exact_int8(y):
    a = y.abs().amax(-1, keepdim=True)
    return torch.round(y * 127 / a.clamp(min=1e-300)) * a / 127


def _exact_e4m3(y):
    a = y.abs().amax(-1, keepdim=True)
    u = y * 448 / a.clamp(min=1e-300)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)  # 3 bits; 2^-9 below 2^-6
    return torch.round(u / step) * step * a / 448


def _exact_cached(s, b, n):
    """The first n cached keys and values of sequence b, (n, Hkv, d)."""
    c, d, Hkv = s["cache"], s["d"], s["Hkv"]
    size = c["ks"].shape[2]
    pages = s["page_table"][b, :-(-n // size)].long()
    k = c["k8"][pages].double() * c["ks"][pages].double()[..., None]
    v = c["v8"][pages].view(torch.float8_e4m3fn).double() * c["vs"][pages].double()[..., None]
    return tuple(x.transpose(1, 2).reshape(-1, Hkv, x.shape[-1])[:n, :, :d] for x in (k, v))


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "norm_rope":
        h = case["rot"] // 2
        row = s["cos_sin"][s["positions"].long()]
        out = {}
        for name in ("q", "k"):
            x = s[name]
            per = [x] if case["layout"] == "packed" else [y if case["layout"] == "NHD" else y.transpose(0, 1) for y in x]
            per = [_exact_rows(y, s[name + "_weight"], case["norm"], row[:, :h], row[:, h:], case["interleaved"]) for y in per]
            out[name] = per[0] if case["layout"] == "packed" else torch.stack(
                [y if case["layout"] == "NHD" else y.transpose(0, 1) for y in per])
        return out
    if case["op"] == "append":
        new, hist = _append_lengths(case)
        cos = sin = None
        if case["rot"]:
            at = torch.cat([torch.arange(a, a + n, device="cuda") for n, a in zip(new, hist)])
            cos, sin = s["cos_sin"][at].chunk(2, -1)
        q = _exact_rows(s["q"], s["q_weight"], case["norm"], cos, sin, case["interleaved"])
        k = _exact_rows(s["k"], s["k_weight"], case["norm"], cos, sin, case["interleaved"])
        mean = 0 if s["k_mean"] is None else s["k_mean"].double()
        return dict(q=q, k=_exact_int8(k - mean) + mean, v=_exact_e4m3(s["v"].double()))
    lens = _lengths(case["B"], case["max_len"], case["ragged"])
    if case["op"] == "gather":
        parts = [_exact_cached(s, b, n) for b, n in enumerate(lens)]
        k, v = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        return dict(k=k if s["k_mean"] is None else k + s["k_mean"].double(), v=v)
    out = torch.zeros((case["B"], case["Hq"], d), dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    for b, n in enumerate(lens):
        if n:
            k, v = _exact_cached(s, b, n)
            q = s["q"][b].double().view(case["Hkv"], G, d)
            score = torch.einsum("hgd,nhd->hgn", q, k) / d ** 0.5
            out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(score, -1), v).reshape(case["Hq"], d)
    return out
