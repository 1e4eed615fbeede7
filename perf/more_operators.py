"""The 8-bit key/value cache and the attention over a shared prefix as measured cases: quantising keys and values as they
enter the pages (their rotation part of the head only, or scaled for long contexts), reading rows back, one-token attention
over the quantised pages, and the attention of a batch whose sequences begin alike.

Each case has a plain form (elementary torch operations in 32 bits, in 64 where angles need them) and the call a program
makes of the library.  ``exact`` gives the same outputs from the definitions in 64 bits.

What the cache holds of a row (one position of one head): codes c in e4m3 and one exponent byte b, for the values
c 2^(b - 127), with the least power of two that keeps the row's largest value within 448; b = 0 is a row of zeros.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
PLAIN, FULL = "plain", dict(layout="interleaved", dims=0, factor=1.0, original=0, low=1.0, high=4.0, magnitude=1.0)


def listed():
    return [
        # one new frame of each of eight sessions, the model's own heads and rotation: latency counts
        dict(name="append8_step", op="append", seqs=8, tokens=8, hq=32, hkv=32, hd=128, page=16, dtype=BF16, far=3000, **FULL),
        # packed prompts of uneven length, grouped heads, half of each head rotated, angles stretched eightfold
        dict(name="append8_prompt", op="append", seqs=7, tokens=8192, hq=32, hkv=8, hd=128, page=16, dtype=BF16, far=65536,
             layout="half", dims=64, factor=8.0, original=8192, low=1.0, high=4.0, magnitude=1.2),
        # one session's whole window leaves the cache, as for a move to another server
        dict(name="read8_session", op="read", seqs=1, len=3000, hkv=32, hd=128, page=64, dtype=BF16, ragged=False),
        # the histories of a batch, for a pass over them in the model's type
        dict(name="read8_batch", op="read", seqs=32, len=8192, hkv=8, hd=128, page=16, dtype=BF16, ragged=True),
        # one session's frame over a full ring's worth of keys
        dict(name="decode8_one", op="decode", seqs=1, len=3000, hq=32, hkv=32, hd=128, page=64, dtype=BF16, window=0, ragged=False),
        # a serving batch of uneven lengths, grouped heads, small pages
        dict(name="decode8_batch", op="decode", seqs=32, len=8192, hq=32, hkv=8, hd=128, page=16, dtype=BF16, window=0, ragged=True),
        # many short contexts, odd groups, queries in the parity type
        dict(name="decode8_short", op="decode", seqs=64, len=1000, hq=24, hkv=8, hd=64, page=48, dtype=F32, window=0, ragged=True),
        # few long contexts: the work has to be split over the length
        dict(name="decode8_long", op="decode", seqs=4, len=131072, hq=64, hkv=8, hd=128, page=128, dtype=BF16, window=0, ragged=True),
        # sessions of one persona: its prompt of 250 frames shared, the model's own heads and window
        dict(name="shared_persona", op="shared", seqs=16, groups=1, prefix=250, own_len=500, hq=32, hkv=32, hd=128, page=2, dtype=BF16,
             cache=PLAIN, window=3000),
        # a batch behind one long system prompt, grouped heads
        dict(name="shared_batch", op="shared", seqs=64, groups=1, prefix=7000, own_len=1000, hq=32, hkv=8, hd=128, page=16, dtype=BF16,
             cache=PLAIN, window=0),
        # three prompts of uneven length and popularity in one batch, over the 8-bit cache
        dict(name="shared_groups", op="shared", seqs=96, groups=3, prefix=6000, own_len=300, hq=32, hkv=8, hd=128, page=16, dtype=BF16,
             cache="e4m3", window=0),
        # a large batch over one long document: products, not bytes, are what it costs
        dict(name="shared_long", op="shared", seqs=256, groups=1, prefix=32768, own_len=200, hq=64, hkv=8, hd=128, page=64, dtype=BF16,
             cache=PLAIN, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "shared", "shared"])
    hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 8])
    while hkv * g > 64:
        hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 8])
    hd, dtype = rng.choice([64, 128]), rng.choice([BF16, BF16, F32])
    page = rng.choice([1, 16, 32, 48, 64, 128])
    if op == "append":
        tokens = _log(rng, 1, 8192)
        if tokens * hkv * (g + 2) * hd * (2 if dtype == BF16 else 4) > 100_000_000:
            tokens = max(1, tokens // 8)
        factor = rng.choice([1.0, 2.0, 8.0])
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 64)), tokens=tokens, hq=hkv * g, hkv=hkv, hd=hd, page=page, dtype=dtype,
                    far=_log(rng, 100, 131072), layout=rng.choice(["interleaved", "half"]), dims=rng.choice([0, 32, 48, hd]), factor=factor,
                    original=0 if factor == 1.0 else rng.choice([0, 4096, 8192]), low=1.0, high=rng.choice([4.0, 32.0]),
                    magnitude=rng.choice([1.0, 1.1]))
    if op == "read":
        seqs, length = _log(rng, 1, 64), _log(rng, 16, 16384)
        while seqs * length * hkv * hd > 60_000_000:
            length = max(16, length // 2)
            seqs = max(1, seqs // 2)
        return dict(op=op, seqs=seqs, len=length, hkv=hkv, hd=hd, page=page, dtype=dtype, ragged=rng.random() < 0.7)
    if op == "decode":
        seqs, length = _log(rng, 1, 64), _log(rng, 16, 65536)
        while 2 * seqs * length * hkv * hd > 600_000_000:
            length = max(16, length // 2)
            seqs = max(1, seqs // 2)
        return dict(op=op, seqs=seqs, len=length, hq=hkv * g, hkv=hkv, hd=hd, page=page, dtype=dtype, window=rng.choice([0, 0, 1000, 3000 - 1]),
                    ragged=rng.random() < 0.7)
    seqs, groups, prefix, own_len = _log(rng, 2, 128), rng.choice([1, 1, 2, 5]), _log(rng, 60, 20000), _log(rng, 1, 1000)
    if dtype == F32:
        prefix, seqs = min(prefix, 5000), min(seqs, 40)
    while seqs * hkv * g * prefix > 64 * 32 * 20000 or seqs * own_len * hkv * hd > 100_000_000:
        seqs = max(2, seqs // 2)
        prefix = max(60, prefix // 2)
    return dict(op=op, seqs=seqs, groups=min(groups, seqs), prefix=prefix, own_len=own_len, hq=hkv * g, hkv=hkv, hd=hd, page=page, dtype=dtype,
                cache=rng.choice([PLAIN, "e4m3"]), window=rng.choice([0, 0, 0, 3000]))


def _lengths(case):
    """Uneven lengths of at least one token, in no order, that add up to the case's tokens."""
    r = np.random.RandomState(case["tokens"])
    n, total = case["seqs"], case["tokens"]
    w = np.linspace(1.0, 4.0, n) if n > 1 else np.ones(1)
    lens = np.maximum(1, np.floor(total * w / w.sum())).astype(np.int64)
    lens[-1] += total - lens.sum()
    while lens[-1] < 1:
        lens[np.argmax(lens)] -= 1
        lens[-1] += 1
    r.shuffle(lens)
    return [int(x) for x in lens]


def _kv_lengths(case):
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [case["len"]] * n
    return [max(1, int(case["len"] * (i + 1) / n) - (i * 7) % 13) for i in range(n)]


def _groups(case):
    """First sequence of each group and the end, prefixes (whole pages), and lengths of all sequences."""
    n, ng, page = case["seqs"], case["groups"], case["page"]
    w = np.cumsum(np.arange(ng, 0, -1))
    first = [0] + [max(i + 1, min(n - (ng - 1 - i), int(round(n * c / w[-1])))) for i, c in enumerate(w)]
    first[-1] = n
    prefix = [max(page, int(case["prefix"] * (i + 2) / (ng + 1)) // page * page) for i in range(ng)]
    lens = []
    for i in range(ng):
        for s in range(first[i], first[i + 1]):
            lens.append(prefix[i] + 1 + (s * 37) % case["own_len"])
    return first, prefix, lens


def _i32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _quantise(x):
    """Codes (float8) and exponent bytes of the rows of x: the least power of two that keeps a row within 448."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    b = torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 127) + 127
    b = torch.where(m == 0, torch.zeros_like(b), b)
    return torch.ldexp(x, (127 - b)[..., None]).to(torch.float8_e4m3fn), b.to(torch.uint8)


def _values(codes, b):
    """What codes (bytes) and exponent bytes stand for, in 32 bits."""
    b = b.int()
    v = torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (b - 127)[..., None])
    return torch.where((b == 0)[..., None], torch.zeros_like(v), v)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, 1.0, generator=gen)

    s = dict(case)
    dt, hkv, hd, page = DT[case["dtype"]], case["hkv"], case["hd"], case["page"]
    hq = s["hq"] = case.get("hq", hkv)

    def pool(pages):
        if case.get("cache") == PLAIN:
            s["kc"], s["vc"] = normal(pages, hkv, page, hd, dtype=dt), normal(pages, hkv, page, hd, dtype=dt)
            return
        for c, b in (("kc", "kb"), ("vc", "vb")):
            s[c] = torch.empty(pages, hkv, page, hd, dtype=torch.uint8, device=dev)
            s[b] = torch.empty(pages, hkv, page, dtype=torch.uint8, device=dev)
            step = max(1, 100_000_000 // (hkv * page * hd))
            for i in range(0, pages, step):
                code, e = _quantise(normal(min(step, pages - i), hkv, page, hd))
                s[c][i:i + step], s[b][i:i + step] = code.view(torch.uint8), e

    def table(need, base=None):
        """A table of distinct pages in a shuffled pool; `base[i]`: (group, pages that the group's sequences share)."""
        groups = {} if base is None else dict(base)
        count = sum(n - (base[i][1] if base else 0) for i, n in enumerate(need)) + sum(groups.values())
        order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
        t = torch.full((len(need), max(need)), -1, dtype=torch.int32, device=dev)
        at, shared = 0, {}
        for g, n in groups.items():
            shared[g] = order[at:at + n]
            at += n
        for i, n in enumerate(need):
            m = 0
            if base is not None:
                m = base[i][1]
                t[i, :m] = shared[base[i][0]]
            t[i, m:n] = order[at:at + n - m]
            at += n - m
        s["table"] = t
        pool(count)

    if case["op"] == "append":
        lens = _lengths(case)
        n = sum(lens)
        past = np.random.RandomState(case["far"]).randint(0, case["far"], len(lens)).tolist()
        total = [a + b for a, b in zip(past, lens)]
        qkv = normal(n, hq + 2 * hkv, hd).to(dt)  # one projection's output: the three parts are strided views of it
        s.update(lens=lens, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_i32(np.cumsum([0] + lens).tolist()), kv_len=_i32(total))
        # the pool holds the pages that the new tokens reach, and the table names only those
        first = [a // page for a in past]
        need = [-(-b // page) - a for a, b in zip(first, total)]
        order = torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32)
        t = torch.full((len(lens), max(-(-b // page) for b in total)), -1, dtype=torch.int32, device=dev)
        at = 0
        for i, c in enumerate(need):
            t[i, first[i]:first[i] + c] = order[at:at + c]
            at += c
        s["table"] = t
        pool(sum(need))
        s["q_out"], s["k_out"] = torch.empty(n, hq, hd, dtype=dt, device=dev), torch.empty(n, hkv, hd, dtype=dt, device=dev)
        # what the cache then holds of the new tokens, in 16 bits, which hold each value exactly
        s["k_back"], s["v_back"] = (torch.empty(n, hkv, hd, dtype=torch.bfloat16, device=dev) for _ in "kv")
    elif case["op"] == "read":
        lens = _kv_lengths(case)
        table([-(-n // page) for n in lens])
        s.update(lens=lens, cu=_i32(np.cumsum([0] + lens).tolist()), kv_len=_i32(lens))
        s["k_back"], s["v_back"] = (torch.empty(sum(lens), hkv, hd, dtype=dt, device=dev) for _ in "kv")
    else:
        if case["op"] == "decode":
            lens = _kv_lengths(case)
            table([-(-n // page) for n in lens])
        else:
            first, prefix, lens = _groups(case)
            base = [(g, prefix[g] // page) for g in range(len(prefix)) for _ in range(first[g], first[g + 1])]
            table([-(-n // page) for n in lens], base)
            s.update(first=first, prefix_lens=prefix, groups_cu=_i32(first), prefix_len=_i32(prefix))
        s.update(lens=lens, kv_len=_i32(lens), q=normal(len(lens), hq, hd, dtype=dt), out=torch.empty(len(lens), hq, hd, dtype=dt, device=dev))
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        if "kb" in s:
            s["cache"] = mfs.QuantKV(s["kc"], s["vc"], s["kb"], s["vb"], s["table"])
        else:
            s["cache"] = mfs.PagedKV(s["kc"], s["vc"], s["table"])
        if case["op"] == "append":
            s["rope"] = mfs.Rope(case["layout"], dims=case["dims"], theta=10000.0, factor=case["factor"], original=case["original"],
                                 low=case["low"], high=case["high"], magnitude=case["magnitude"])
        elif case["op"] == "decode":
            s["workspace"] = mfs.mfs_paged_attention_workspace(s["cache"], hq)
        elif case["op"] == "shared":
            s["workspace"] = mfs.mfs_shared_attention_workspace(s["cache"], hq, len(lens))
    return s


def run(state):
    return {"append": _append, "read": _read, "decode": _decode, "shared": _shared}[state["op"]](state)


def _positions(s, n):
    """Sequence and position of each of n packed rows: the last ones of each sequence."""
    tok = torch.arange(n, device="cuda")
    seq = torch.bucketize(tok, s["cu"][1:].long(), right=True)
    return seq, s["kv_len"].long()[seq] - s["cu"].long()[seq + 1] + tok


def _append(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_kv_append(s["cache"], s["k"], s["v"], s["cu"], s["kv_len"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"], rope=s["rope"])
        mfs.mfs_kv_read(s["cache"], s["cu"], s["kv_len"], s["k_back"], s["v_back"])
        return s["q_out"], s["k_out"], s["k_back"], s["v_back"]
    dims = s["dims"] or s["hd"]
    seq, pos = _positions(s, s["k"].shape[0])
    turns = 10000.0 ** (-2.0 * torch.arange(dims // 2, device="cuda", dtype=torch.float64) / dims) / (2 * math.pi)
    kept = (turns * s["original"] - s["low"]) / (s["high"] - s["low"]) if s["original"] else torch.zeros_like(turns)
    kept = kept.clamp(0.0, 1.0)
    angle = pos.double()[:, None] * (turns * (kept + (1.0 - kept) / s["factor"])) * (2 * math.pi)
    c, sn = (torch.cos(angle) * s["magnitude"]).float()[:, None], (torch.sin(angle) * s["magnitude"]).float()[:, None]

    def rotate(x):
        x = x.float()
        r = x[..., :dims]
        if s["layout"] == "half":
            a, b = r.chunk(2, dim=-1)
            r = torch.cat([a * c - b * sn, a * sn + b * c], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
        return torch.cat([r, x[..., dims:]], -1)

    page, row = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    k = rotate(s["k"])
    s["q_out"].copy_(rotate(s["q"]).to(s["q"].dtype))
    s["k_out"].copy_(k.to(s["k"].dtype))
    kc, kb = _quantise(k)
    vc, vb = _quantise(s["v"])
    s["kc"][page, :, row], s["kb"][page, :, row] = kc.view(torch.uint8), kb
    s["vc"][page, :, row], s["vb"][page, :, row] = vc.view(torch.uint8), vb
    s["k_back"].copy_(_values(s["kc"][page, :, row], s["kb"][page, :, row]).bfloat16())
    s["v_back"].copy_(_values(s["vc"][page, :, row], s["vb"][page, :, row]).bfloat16())
    return s["q_out"], s["k_out"], s["k_back"], s["v_back"]


def _read(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_kv_read(s["cache"], s["cu"], s["kv_len"], s["k_back"], s["v_back"])
        return s["k_back"], s["v_back"]
    seq, pos = _positions(s, s["k_back"].shape[0])
    page, row = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    s["k_back"].copy_(_values(s["kc"][page, :, row], s["kb"][page, :, row]).to(s["k_back"].dtype))
    s["v_back"].copy_(_values(s["vc"][page, :, row], s["vb"][page, :, row]).to(s["v_back"].dtype))
    return s["k_back"], s["v_back"]


def _rows(s, which, page, row):
    """Keys or values at pages and rows, in 32 bits."""
    if "kb" in s:
        return _values(s[which + "c"][page, :, row], s[which + "b"][page, :, row])
    return s[which + "c"][page, :, row].float()


def _decode(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_paged_attention(s["cache"], s["q"], s["kv_len"], s["out"], window=s["window"], workspace=s["workspace"])
        return s["out"]
    n, hkv, hd = len(s["lens"]), s["hkv"], s["hd"]
    first = max(0, min(s["lens"]) - s["window"]) if s["window"] else 0
    pos = torch.arange(first, max(s["lens"]), device="cuda")
    length = s["kv_len"].long()[:, None]
    seen = pos[None] < length
    if s["window"]:
        seen = seen & (pos[None] >= length - s["window"])
    page = s["table"].long()[:, pos // s["page"]].clamp(min=0)
    row = (pos % s["page"])[None].expand_as(page)
    q = s["q"].float().view(n, hkv, -1, hd)
    a = torch.matmul(q, _rows(s, "k", page, row).permute(0, 2, 3, 1)) * (1.0 / math.sqrt(hd))
    seen = seen[:, None, None]
    a = torch.where(seen, a, torch.full_like(a, -math.inf))
    a = torch.where(seen, torch.exp(a - a.amax(-1, keepdim=True)), torch.zeros_like(a))
    a = a / a.sum(-1, keepdim=True)
    return torch.matmul(a, _rows(s, "v", page, row).permute(0, 2, 1, 3)).reshape(n, -1, hd).to(s["q"].dtype)


def _shared(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_shared_attention(s["cache"], s["q"], s["kv_len"], s["groups_cu"], s["prefix_len"], s["out"], window=s["window"],
                                 workspace=s["workspace"])
        return s["out"]
    n, hkv, hd, ps = len(s["lens"]), s["hkv"], s["hd"], s["page"]
    g, scale = s["hq"] // hkv, 1.0 / math.sqrt(hd)
    first, prefix = s["groups_cu"].long(), s["prefix_len"].long()
    seq = torch.arange(n, device="cuda")
    grp = torch.bucketize(seq, first[1:], right=True)
    length, least = s["kv_len"].long(), s["kv_len"].long() - (s["window"] or (1 << 40))  # the first position a sequence sees
    # the prefixes, once a group; the group's sequences side by side, a short group padded with its first
    most = max(b - a for a, b in zip(s["first"], s["first"][1:]))
    place = first[:-1, None] + torch.arange(most, device="cuda")
    inside = place < first[1:, None]
    place = torch.where(inside, place, first[:-1, None])
    pos = torch.arange(max(s["prefix_lens"]), device="cuda")
    page = s["table"].long()[first[:-1]][:, (pos // ps).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    row = (pos % ps)[None].expand_as(page)
    q = s["q"].float().view(n, hkv, g, hd)
    qg = q[place].permute(0, 2, 1, 3, 4).reshape(len(prefix), hkv, most * g, hd)
    a = torch.matmul(qg, _rows(s, "k", page, row).permute(0, 2, 3, 1)) * scale
    a = a.view(len(prefix), hkv, most, g, -1).permute(0, 2, 1, 3, 4)[grp, seq - first[grp]]
    seen = (pos[None] < prefix[grp][:, None]) & (pos[None] < length[:, None]) & (pos[None] >= least[:, None])
    a = torch.where(seen[:, None, None], a, a.new_full((), -math.inf))
    # what follows the prefix, each sequence's own
    at = torch.arange(max(l - s["prefix_lens"][i] for i, f in enumerate(s["first"][:-1]) for l in s["lens"][f:s["first"][i + 1]]), device="cuda")
    at = prefix[grp][:, None] + at[None]
    mine = (at < length[:, None]) & (at >= least[:, None])
    at = torch.minimum(at, length[:, None] - 1)
    page1, row1 = s["table"].long().gather(1, at // ps).clamp(min=0), at % ps
    b = torch.matmul(q, _rows(s, "k", page1, row1).permute(0, 2, 3, 1)) * scale
    b = torch.where(mine[:, None, None], b, b.new_full((), -math.inf))
    top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a, b = torch.exp(a - top), torch.exp(b - top)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = torch.matmul(b, _rows(s, "v", page1, row1).permute(0, 2, 1, 3))
    wg = a[place].permute(0, 2, 1, 3, 4).reshape(len(prefix), hkv, most * g, -1)
    og = torch.matmul(wg, _rows(s, "v", page, row).permute(0, 2, 1, 3)).view(len(prefix), hkv, most, g, hd)
    o = o + og.permute(0, 2, 1, 3, 4)[grp, seq - first[grp]]
    return (o / total).reshape(n, -1, hd).to(s["q"].dtype)


def work(case):
    e, hkv, hd = (2 if case["dtype"] == BF16 else 4), case["hkv"], case["hd"]
    if case["op"] == "append":  # q in and out; k in, out and back; v in and back; codes written and read
        n, hq = case["tokens"], case["hq"]
        return {"bytes": n * (hd * (e * (2 * hq + 3 * hkv) + 4 * hkv) + 4 * hkv * (hd + 1)), "flops": 3 * n * hd * (hq + hkv)}
    if case["op"] == "read":
        return {"bytes": 2 * sum(_kv_lengths(case)) * hkv * (hd + 1 + hd * e), "flops": 2 * sum(_kv_lengths(case)) * hkv * hd}
    hq, w = case["hq"], case["window"]
    if case["op"] == "decode":
        keys = sum(min(n, w) if w else n for n in _kv_lengths(case))
        return {"bytes": 2 * keys * hkv * (hd + 1) + 2 * e * hd * case["seqs"] * hq + 4 * case["seqs"], "flops": 4 * keys * hq * hd}
    first, prefix, lens = _groups(case)
    per = 2 * hkv * (hd * e if case["cache"] == PLAIN else hd + 1)
    pairs = sum(min(n, w) if w else n for n in lens)
    keys = 0
    for i, p in enumerate(prefix):
        seen = [(max(0, n - w) if w else 0, n) for n in lens[first[i]:first[i + 1]]]
        keys += max(0, p - min(a for a, _ in seen)) + sum(n - max(p, a) for a, n in seen)
    return {"bytes": keys * per + 2 * e * hd * len(lens) * hq + 4 * len(lens), "flops": 4 * pairs * hq * hd}


def _exact_e4m3(x):
    """The nearest values of the rows of x (64 bits) in the cache's form: four significant bits under a power of two."""
    top = np.abs(x).max(-1, keepdims=True)
    e = np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0))
    e = np.where(top > 448.0 * np.exp2(e), e + 1, np.where(top <= 448.0 * np.exp2(e - 1), e - 1, e))
    y = x / np.exp2(e)
    step = np.exp2(np.maximum(np.floor(np.log2(np.where(y != 0, np.abs(y), 1.0))), -6.0) - 3.0)
    return np.rint(y / step) * step * np.exp2(e)


def _exact_values(codes, b):
    """Bytes as sign, four bits of exponent and three of fraction, under 2^(b - 127)."""
    table = np.array([(-1.0 if c & 128 else 1.0) * ((8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10) if c & 120 else (c & 7) * 2.0 ** -9)
                      for c in range(256)])
    size = np.where(np.arange(256) > 0, np.exp2(np.arange(256) - 127.0), 0.0)
    return torch.from_numpy(table).cuda()[codes.int()] * torch.from_numpy(size).cuda()[b.int()][..., None]


def exact(case, seed):
    s = prepare(case, seed)
    hd, hkv, page = case["hd"], case["hkv"], case["page"]
    if case["op"] == "append":
        q, k, v = (s[x].cpu().double().numpy() for x in "qkv")
        dims = case["dims"] or hd
        i = np.arange(dims // 2)
        x, y = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + dims // 2)
        freq = np.power(10000.0, -2.0 * i / dims)
        if case["original"]:
            in_all = case["original"] * freq / (2 * np.pi)  # turns over the original length
            part = np.clip((in_all - case["low"]) / (case["high"] - case["low"]), 0, 1)
            freq = part * freq + (1 - part) * freq / case["factor"]
        else:
            freq = freq / case["factor"]
        at = np.concatenate([np.arange(n - c, n) for n, c in zip(s["kv_len"].tolist(), s["lens"])])
        turn = case["magnitude"] * np.exp(1j * at[:, None] * freq)[:, None]

        def turned(a):
            z, out = (a[..., x] + 1j * a[..., y]) * turn, a.copy()
            out[..., x], out[..., y] = z.real, z.imag
            return out

        kr = turned(k)
        return turned(q), kr, _exact_e4m3(kr), _exact_e4m3(v)
    dev = "cuda"
    if "kb" in s:
        kc, vc = _exact_values(s["kc"], s["kb"]), _exact_values(s["vc"], s["vb"])
    else:
        kc, vc = s["kc"], s["vc"]

    def history(i, a, b):
        at = torch.arange(a, b, device=dev)
        pages = s["table"][i].long()[at // page]
        return kc[pages, :, at % page].double(), vc[pages, :, at % page].double()

    if case["op"] == "read":
        got = [history(i, 0, n) for i, n in enumerate(s["lens"])]
        return torch.cat([k for k, _ in got]), torch.cat([v for _, v in got])
    hq, w = case["hq"], case["window"]
    g, scale = hq // hkv, 1.0 / math.sqrt(hd)
    out = torch.empty(len(s["lens"]), hq, hd, dtype=torch.float64, device=dev)
    for i, n in enumerate(s["lens"]):
        k, v = history(i, max(0, n - w) if w else 0, n)
        q = s["q"][i].double().view(hkv, g, hd)
        a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) * scale, -1)
        out[i] = torch.einsum("hgl,lhd->hgd", a, v).reshape(hq, hd)
    return out
