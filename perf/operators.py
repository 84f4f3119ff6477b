"""Measured cases of the operators that bring new tokens into a paged FP8 cache and attend over it.

Three operators that a serving loop runs one after the other on a ragged batch of new tokens
(token i of sequence b sits at position ctx_lens[b] + i):

  norm    pw_qk_norm_rope  RMS norm of every query and key head and the position rotation
  append  pw_append        norm and rotation of the keys on the way into the E4M3 pages; values too
  attn    pw_chunk_attn    causal attention of the new tokens over the paged E4M3 cache

A case's lengths follow from its numbers alone (see `lengths`); the values follow from the seed.
"""
import math

import torch

own = False

PAGE, DIM = 64, 128
EPS = 1e-6
BASE = 10000.0
SCALE = 1.0 / 64.0  # cache scale: codes of unit-variance keys use the middle of the E4M3 range


def listed():
    return [
        # one user's next token: the call's latency
        dict(name="attn decode 1 x 2k", op="attn", B=1, q=1, q_min=1, ctx=2047, ctx_min=2047, Hq=32, Hkv=8, window=0, lse=False),
        # a serving batch of single tokens, contexts of every length
        dict(name="attn decode 64 ragged", op="attn", B=64, q=1, q_min=1, ctx=16383, ctx_min=500, Hq=64, Hkv=8, window=0, lse=False),
        # few users with contexts as long as the cache allows
        dict(name="attn decode 4 x 128k", op="attn", B=4, q=1, q_min=1, ctx=131071, ctx_min=131071, Hq=64, Hkv=8, window=0, lse=False),
        # a few drafted tokens of each user checked at once
        dict(name="attn verify 32 x 5", op="attn", B=32, q=5, q_min=5, ctx=8191, ctx_min=1000, Hq=32, Hkv=8, window=0, lse=True),
        # chunks of several prompts in one step, a sliding window, one user already decoding
        dict(name="attn chunks ragged", op="attn", B=5, q=911, q_min=1, ctx=12001, ctx_min=0, Hq=32, Hkv=8, window=4096, lse=False),
        # a large chunk late in a long prompt: the step that a long prefill is made of
        dict(name="attn chunk 2k at 32k", op="attn", B=1, q=2048, q_min=2048, ctx=30720, ctx_min=30720, Hq=64, Hkv=8, window=0, lse=True),
        # queries and keys of one decoding step
        dict(name="norm decode 64", op="norm", B=64, q=1, q_min=1, ctx=16383, ctx_min=500, Hq=64, Hkv=8, norm=True, rot=128, interleaved=False),
        # chunks of several prompts, half of each head rotated in neighbouring pairs
        dict(name="norm chunks ragged", op="norm", B=7, q=2003, q_min=1, ctx=9000, ctx_min=0, Hq=32, Hkv=8, norm=True, rot=64, interleaved=True),
        # one prompt from its start
        dict(name="norm prompt 16k", op="norm", B=1, q=16384, q_min=16384, ctx=0, ctx_min=0, Hq=64, Hkv=8, norm=True, rot=128, interleaved=False),
        # one decoding step of a serving batch
        dict(name="append decode 64", op="append", B=64, q=1, q_min=1, ctx=16383, ctx_min=500, Hq=64, Hkv=8, norm=True, rot=128, interleaved=False),
        # chunks of several prompts, pages that end inside a chunk, no key norm
        dict(name="append chunks ragged", op="append", B=9, q=1501, q_min=1, ctx=7001, ctx_min=0, Hq=32, Hkv=8, norm=False, rot=64, interleaved=True),
        # two long prompts from their starts
        dict(name="append prompts 2 x 16k", op="append", B=2, q=16384, q_min=16384, ctx=0, ctx_min=0, Hq=64, Hkv=8, norm=True, rot=128, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hq, Hkv = rng.choice([(8, 1), (8, 2), (32, 8), (64, 8), (16, 16), (24, 8)])
    op = rng.choice(["attn", "attn", "norm", "append"])
    if op == "attn":
        kind = rng.choice(["decode", "verify", "chunk"])
        if kind == "chunk":
            B, q = rng.randint(1, 6), _log_int(rng, 17, 2048)
            q_min, ctx = rng.randint(1, q), _log_int(rng, 1, 30000)
        else:
            B, q = _log_int(rng, 1, 64), 1 if kind == "decode" else rng.randint(2, 8)
            q_min, ctx = rng.randint(1, q), _log_int(rng, 1, 130000)
        # no more work or room than the largest listed cases take
        while B > 1 and (B * q * (ctx + q) * Hq > 2048 * 32768 * 64 or B * (ctx + q) * Hkv > 64 * 16384 * 8):
            B -= 1
        if B * q * (ctx + q) * Hq > 2048 * 32768 * 64:
            q = max(1, 2048 * 32768 * 64 // ((ctx + q) * Hq))
            q_min = min(q_min, q)
        window = rng.choice([0, 0, rng.randint(1, ctx + q)])
        return dict(op=op, B=B, q=q, q_min=q_min, ctx=ctx, ctx_min=rng.randint(0, ctx), Hq=Hq, Hkv=Hkv, window=window, lse=rng.random() < 0.5)
    B = _log_int(rng, 1, 64)
    q = _log_int(rng, 1, 16384)
    while B > 1 and B * q > (16384 if op == "norm" else 32768):
        B = (B + 1) // 2
    ctx = rng.choice([0, _log_int(rng, 1, 30000)])
    return dict(op=op, B=B, q=q, q_min=rng.randint(1, q), ctx=ctx, ctx_min=rng.randint(0, ctx), Hq=Hq, Hkv=Hkv, norm=rng.random() < 0.6,
                rot=rng.choice([128, 128, 64, 32]), interleaved=rng.random() < 0.4)


def lengths(case):
    """New tokens and context tokens of each sequence: spread from the least to the most, both ends taken, in a mixed order."""
    B = case["B"]

    def spread(lo, hi, step):
        return [hi if B == 1 else lo + (hi - lo) * ((i * step) % B) // (B - 1) for i in range(B)]

    step = next(s for s in (7, 11, 13, 17, 19, 1) if math.gcd(s, B) == 1)
    return spread(case["q_min"], case["q"], 1), spread(case["ctx_min"], case["ctx"], step)


def _codes(shape, g, dev):
    """E4M3 codes of unit-variance values at the cache's scale."""
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
    return x.mul_(1.0 / SCALE).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _inputs(case, seed):
    """The inputs of a case, as tensors on the GPU."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ql, cl = lengths(case)
    B, T, Hq, Hkv = case["B"], sum(ql), case["Hq"], case["Hkv"]
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    s = dict(T=T, cu=torch.tensor(cu, dtype=torch.int32, device=dev), ctx=torch.tensor(cl, dtype=torch.int32, device=dev))
    if case["op"] == "attn":
        # heads differ in how sharply they attend
        sharp = torch.linspace(0.5, 3.0, Hq, device=dev)[:, None]
        s["Q"] = (torch.randn((T, Hq, DIM), generator=g, device=dev) * sharp).to(torch.bfloat16)
    else:
        # the packed projection of a layer: queries, keys and values of a token side by side
        qkv = torch.randn((T, Hq + 2 * Hkv, DIM), generator=g, device=dev).to(torch.bfloat16)
        s["Q"], s["K"], s["V"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        for w in ("qw", "kw"):
            s[w] = (1.0 + 0.2 * torch.randn((DIM,), generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
    if case["op"] != "norm":
        pages = [(c + n + PAGE - 1) // PAGE for c, n in zip(cl, ql)]
        n_phys = sum(pages) + 3
        perm = torch.randperm(n_phys, generator=g, device=dev).to(torch.int32)
        s["table"] = torch.full((B, max(pages)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(pages):
            s["table"][b, :n] = perm[at:at + n]
            at += n
        s["K_pages"] = _codes((n_phys, Hkv, PAGE, DIM), g, dev)
        s["V_pages"] = _codes((n_phys, Hkv, PAGE, DIM), g, dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dev = s["cu"].device
    s.update(case=case, status=torch.zeros(1, dtype=torch.int32, device=dev))
    T, Hq, Hkv = s["T"], case["Hq"], case["Hkv"]
    if case["op"] == "attn":
        s["O"] = torch.empty((T, Hq, DIM), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev) if case["lse"] else None
        if own:
            from dynamic_sparse_attention_pw_b200 import api
            s["workspace"] = api.chunk_workspace(case["B"], T, Hq, Hkv, max_q_len=case["q"], device=dev)
    else:
        # the rotation's table is made once for a model: cos | sin of every position, angles in 64 bits
        n = case["ctx"] + case["q"]
        inv = BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
        angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["op"] == "norm":
            s["Q_out"] = torch.empty((T, Hq, DIM), dtype=torch.bfloat16, device=dev)
            s["K_out"] = torch.empty((T, Hkv, DIM), dtype=torch.bfloat16, device=dev)
    return s


def _places(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["T"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b] + s["ctx"].long()[b]


def _norm_rope(x, weight, pos, table, rot, interleaved):
    """x [T, H, 128] -> its heads normalised (where a weight is given) and rotated, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    cos, sin = table[pos][:, None, :].split(rot // 2, -1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_norm(s):
    c, (_, pos) = s["case"], _places(s)
    return (_norm_rope(s["Q"], s["qw"], pos, s["rope"], c["rot"], c["interleaved"]).to(torch.bfloat16),
            _norm_rope(s["K"], s["kw"], pos, s["rope"], c["rot"], c["interleaved"]).to(torch.bfloat16))


def _plain_append(s):
    c, (b, pos) = s["case"], _places(s)
    k = _norm_rope(s["K"], s["kw"], pos, s["rope"], c["rot"], c["interleaved"])
    page = s["table"].long()[b, pos // PAGE]
    for pages, x in ((s["K_pages"], k), (s["V_pages"], s["V"].float())):
        pages[page, :, pos % PAGE] = (x / SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return s["K_pages"].view(torch.float8_e4m3fn), s["V_pages"].view(torch.float8_e4m3fn)


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    (b, pos), dev = _places(s), s["cu"].device
    row = pos - s["ctx"].long()[b]  # token's number in its chunk
    Q = torch.zeros((B, c["q"], Hq, DIM), device=dev)
    Q[b, row] = s["Q"].float() * (SCALE / math.sqrt(DIM))
    Q = Q.view(B, c["q"], Hkv, Hq // Hkv, DIM).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, DIM)

    def dense(pages):  # [B, Hkv, keys, 128]
        x = pages.view(torch.float8_e4m3fn)[s["table"].long().clamp(min=0)].float()
        return x.transpose(1, 2).reshape(B, Hkv, -1, DIM)

    S = torch.matmul(Q, dense(s["K_pages"]).transpose(2, 3)).view(B, Hq, c["q"], -1)
    key = torch.arange(S.shape[-1], device=dev)
    at = s["ctx"].long()[:, None] + torch.arange(c["q"], device=dev)  # position of each query row
    off = key > at[..., None]
    if c["window"]:
        off |= key <= at[..., None] - c["window"]
    S.masked_fill_(off[:, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    S.sub_(m).exp_()
    total = S.sum(-1, keepdim=True)
    O = torch.matmul(S.view(B, Hkv, -1, S.shape[-1]), dense(s["V_pages"])).view(B, Hq, c["q"], DIM)
    O = (O * (SCALE / total)).to(torch.bfloat16)
    lse = (m + total.log()).squeeze(-1)
    return (O[b, :, row], lse[b, :, row]) if c["lse"] else O[b, :, row]


def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn}[c["op"]](s)
    from dynamic_sparse_attention_pw_b200 import api
    if c["op"] == "norm":
        return api.pw_qk_norm_rope(s["Q"], s["K"], s["cu"], s["ctx"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rope=s["rope"],
                                   interleaved=c["interleaved"], Q_out=s["Q_out"], K_out=s["K_out"], status=s["status"])
    if c["op"] == "append":
        api.pw_append(s["K"], s["V"], s["K_pages"], s["V_pages"], s["table"], s["cu"], s["ctx"], k_scale=SCALE, v_scale=SCALE,
                      k_weight=s["kw"], eps=EPS, rope=s["rope"], interleaved=c["interleaved"], status=s["status"])
        return s["K_pages"].view(torch.float8_e4m3fn), s["V_pages"].view(torch.float8_e4m3fn)
    api.pw_chunk_attn(s["Q"], s["K_pages"], s["V_pages"], s["table"], s["cu"], s["ctx"], max_q_len=c["q"], k_scale=SCALE, v_scale=SCALE,
                      window=c["window"], O=s["O"], lse=s["lse"], workspace=s["workspace"], status=s["status"])
    return (s["O"], s["lse"]) if c["lse"] else s["O"]


def work(case):
    ql, cl = lengths(case)
    T, Hq, Hkv = sum(ql), case["Hq"], case["Hkv"]
    if case["op"] == "norm":
        n = T * (Hq + Hkv) * DIM
        return {"bytes": 2 * 2 * n + 4 * case["rot"] * (case["ctx"] + case["q"] if T > case["ctx"] + case["q"] else T), "flops": 10 * n}
    if case["op"] == "append":
        n = T * Hkv * DIM
        return {"bytes": 2 * (2 * n + n) + 4 * case["rot"] * (case["ctx"] + case["q"] if T > case["ctx"] + case["q"] else T), "flops": 12 * n}
    w = case["window"]
    read = pairs = 0
    for n, c in zip(ql, cl):
        first = max(0, c + 1 - w) if w else 0  # the first key that any of the chunk's tokens sees
        read += c + n - first
        full = n if not w else max(0, min(n, w - c - 1))  # tokens that see every earlier key
        pairs += full * (c + 1) + full * (full - 1) // 2 + (n - full) * w
    return {"bytes": 2 * read * Hkv * DIM + 2 * 2 * T * Hq * DIM + (4 * T * Hq if case["lse"] else 0), "flops": 4 * pairs * Hq * DIM}


def _exact_heads(x, weight, angle, interleaved):
    """Norm and rotation in 64 bits, by complex numbers: a pair times e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / DIM + EPS).sqrt() * weight.double()
    half = angle.shape[1]
    if interleaved:
        z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half])
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    turned = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _e4m3_values(dev):
    """The value of each of the 256 codes, from the format's definition."""
    code = torch.arange(256, device=dev)
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = torch.where((code & 127) == 127, torch.nan, v)
    return torch.where(code >= 128, -v, v)


def exact(case, seed):
    s = _inputs(case, seed)
    dev = s["cu"].device
    ql, cl = lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    value = _e4m3_values(dev)
    if case["op"] != "attn":
        pos = torch.cat([torch.arange(c, c + n, dtype=torch.float64, device=dev) for n, c in zip(ql, cl)])
        angle = pos[:, None] / BASE ** (torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev) * 2 / case["rot"])
        k = _exact_heads(s["K"], s["kw"], angle, case["interleaved"])
        if case["op"] == "norm":
            return _exact_heads(s["Q"], s["qw"], angle, case["interleaved"]), k
        out = []
        for pages, x in ((s["K_pages"], k), (s["V_pages"], s["V"].double())):
            y, at = value[pages.int()], 0
            for b, (n, c) in enumerate(zip(ql, cl)):
                p = torch.arange(c, c + n, device=dev)
                y[s["table"][b].long()[p // PAGE], :, p % PAGE] = (x[at:at + n] / SCALE).clamp(-448, 448)
                at += n
            out.append(y)
        return tuple(out)
    G = Hq // Hkv
    O = torch.empty((s["T"], Hq, DIM), dtype=torch.float64, device=dev)
    lse = torch.empty((s["T"], Hq), dtype=torch.float64, device=dev)
    at = 0
    for b, (n, c) in enumerate(zip(ql, cl)):
        pages = s["table"][b, :(c + n + PAGE - 1) // PAGE].long()
        i = torch.arange(c, c + n, device=dev)[:, None, None]
        j = torch.arange(c + n, device=dev)
        seen = (j <= i) & (j > i - case["window"]) if case["window"] else j <= i
        for h in range(Hkv):
            k = value[s["K_pages"][pages, h].int()].reshape(-1, DIM)[:c + n] * SCALE
            v = value[s["V_pages"][pages, h].int()].reshape(-1, DIM)[:c + n] * SCALE
            x = (s["Q"][at:at + n, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(DIM)
            x = x.masked_fill_(~seen, -math.inf)
            z = torch.logsumexp(x, -1)
            O[at:at + n, h * G:(h + 1) * G] = x.sub_(z[..., None]).exp_() @ v
            lse[at:at + n, h * G:(h + 1) * G] = z
        at += n
    return (O, lse) if case["lse"] else O
