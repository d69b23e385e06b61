"""The cases of the paged serving step's operators: page tables and slot maps built
on the GPU from request lengths, rotary positions with several axes applied while
new keys and values are stored into pages, attention of one new token over a paged
cache whose lengths live on the device, and cross attention of ragged queries to
paged encoder states.

``run`` computes a case either in its plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the package's entry points; ``exact``
gives the same outputs from the definitions in 64 bits.  Pages hold 64 tokens; a pool
is [slot][kv_heads][64][head_dim].
"""
import random

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
NINF = float("-inf")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 running requests: a token each, a page now and then
        {"op": "tables", "name": "tables_step_64", "n_req": 64, "lo": 100, "hi": 8000, "grow": 0.0, "chunk": 1,
         "gone": 0.0, "max_pages": 256, "short": 0.0},
        # a busy scheduler step: prompt chunks, single tokens and finished requests together
        {"op": "tables", "name": "tables_mixed_1000", "n_req": 1000, "lo": 1, "hi": 30000, "grow": 0.25, "chunk": 600,
         "gone": 0.1, "max_pages": 512, "short": 0.0},
        # the step of a small decode batch far into its history (the repository's head layout)
        {"op": "rope", "name": "rope_step_16", "tokens": 16, "pad": 0, "H": 4, "G": 8, "D": 256, "rot": 256, "axes": 1,
         "pairs": False, "far": 131072, "dtype": "bf16"},
        # a video prompt: time, height and width positions
        {"op": "rope", "name": "rope_video_8200", "tokens": 8200, "pad": 0, "H": 8, "G": 4, "D": 128, "rot": 128,
         "axes": 3, "pairs": False, "far": 2000, "dtype": "bf16"},
        # a padded batch, half of each head rotated in neighbouring pairs
        {"op": "rope", "name": "rope_partial_1001", "tokens": 1001, "pad": 23, "H": 12, "G": 1, "D": 64, "rot": 32,
         "axes": 1, "pairs": True, "far": 5000, "dtype": "f16"},
        # one user's first answer tokens: latency
        {"op": "decode", "name": "decode_one_short", "n_req": 1, "lo": 200, "hi": 200, "empty": 0, "window": 0, "H": 4,
         "G": 8, "D": 256, "dtype": "bf16"},
        # one long context (the repository's 128K history, all in 16 bits)
        {"op": "decode", "name": "decode_one_128k", "n_req": 1, "lo": 131072, "hi": 131072, "empty": 0, "window": 0,
         "H": 4, "G": 8, "D": 256, "dtype": "bf16"},
        # the repository's 16 requests of 8K to 64K tokens
        {"op": "decode", "name": "decode_batch_16", "n_req": 16, "lo": 8192, "hi": 65536, "empty": 0, "window": 0,
         "H": 4, "G": 8, "D": 256, "dtype": "bf16"},
        # many short chats, idle slots of the batch among them, odd head groups, a sliding window
        {"op": "decode", "name": "decode_window_96", "n_req": 96, "lo": 1, "hi": 6000, "empty": 5, "window": 1000,
         "H": 8, "G": 5, "D": 128, "dtype": "f16"},
        # a few decoder tokens against short encodings
        {"op": "cross", "name": "cross_short_4", "n_req": 4, "qlo": 3, "qhi": 9, "slo": 150, "shi": 1500, "clips": 0,
         "H": 8, "G": 2, "D": 64, "dtype": "f16"},
        # text prompts against image encodings
        {"op": "cross", "name": "cross_prompt_8", "n_req": 8, "qlo": 300, "qhi": 1500, "slo": 1601, "shi": 6404,
         "clips": 0, "H": 8, "G": 4, "D": 128, "dtype": "bf16"},
        # each token sees the clip before it and none before the first; the repository's head layout
        {"op": "cross", "name": "cross_clips_3", "n_req": 3, "qlo": 200, "qhi": 900, "slo": 900, "shi": 5000,
         "clips": 4, "H": 4, "G": 8, "D": 256, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["tables", "rope", "decode", "decode", "cross", "cross"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "tables":
        return {"op": op, "n_req": _log(rng, 1, 1000), "lo": 1, "hi": _log(rng, 50, 30000), "grow": rng.choice([0.0, 0.2]),
                "chunk": _log(rng, 1, 600), "gone": rng.choice([0.0, 0.15]), "max_pages": 512 + rng.randrange(40),
                "short": rng.choice([0.0, 0.0, 0.5])}
    if op == "rope":
        D = rng.choice([64, 128, 256])
        H = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 8192 * 128 // D), "pad": rng.choice([0, 0, 7]), "H": H,
                "G": rng.choice([1, 2, 3, 4]), "D": D, "rot": rng.choice([D, D, D // 2]), "axes": rng.choice([1, 3]),
                "pairs": rng.random() < 0.4, "far": _log(rng, 100, 1000000), "dtype": dtype}
    D = rng.choice([64, 128, 256])
    G = rng.choice([1, 2, 4, 5, 8, 8])
    if op == "decode":
        n = _log(rng, 1, 64)
        hi = _log(rng, 64, min(131072, 480000 // n))
        return {"op": op, "n_req": n, "lo": max(1, hi // rng.choice([1, 8, 1000])), "hi": hi, "empty": rng.choice([0, n // 8]),
                "window": rng.choice([0, 0, 500]), "H": rng.choice([1, 2, 4, 8]) if D < 256 else rng.choice([1, 2, 4]), "G": G, "D": D,
                "dtype": dtype}
    n = rng.randint(1, 6)
    qhi = _log(rng, 1, 1200)
    shi = _log(rng, 10, 6000)
    return {"op": op, "n_req": n, "qlo": max(1, qhi // 4), "qhi": qhi, "slo": max(1, shi // 5), "shi": shi,
            "clips": rng.choice([0, 0, 3]), "H": rng.choice([1, 2, 4, 8]) if D < 256 else rng.choice([1, 2, 4]),
            "G": rng.choice([1, 2, 4]), "D": D, "dtype": dtype}


# -------------------------------------------- lengths, fixed by the case alone
def _lengths(case):
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "decode":
        lens = [0 if i < case["empty"] else rng.randint(case["lo"], case["hi"]) for i in range(case["n_req"])]
        rng.shuffle(lens)
        return lens
    if case["op"] == "cross":
        return ([rng.randint(case["qlo"], case["qhi"]) for _ in range(case["n_req"])],
                [rng.randint(case["slo"], case["shi"]) for _ in range(case["n_req"])])
    old, new = [], []
    for _ in range(case["n_req"]):
        a = _log(rng, case["lo"], case["hi"])
        old.append(a)
        if rng.random() < case["gone"]:
            new.append(0 if rng.random() < 0.7 else rng.randint(0, a))  # finished, or a draft taken back
        elif rng.random() < case["grow"]:
            new.append(a + rng.randint(1, case["chunk"]))
        else:
            new.append(a + 1)
    return old, new


def _ranges(case):
    """kv_range of each query token of a case with clips (None without): the clips cut
    the states evenly, a token sees the last clip before it, the first tokens none."""
    if not case["clips"]:
        return None
    q, s = _lengths(case)
    out = []
    for nq, ns in zip(q, s):
        c = case["clips"]
        for i in range(nq):
            k = i * (c + 1) // nq  # 0: before the first clip
            out.append((0, 0) if k == 0 else (ns * (k - 1) // c, ns * k // c))
    return out


def _visible(case, n):
    return min(n, case["window"]) if case["window"] else n


def work(case):
    if case["op"] == "tables":
        old, new = _lengths(case)
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        pages = sum(abs(-(-b // PAGE) + (-a // PAGE)) for a, b in zip(old, new))
        return {"bytes": 16 * tokens + 8 * pages + 24 * case["n_req"], "flops": 4 * tokens}
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": t * ((2 * H * G + 4 * H) * D * 2 + 4 * case["axes"] + 8), "flops": 3 * t * (H * G + H) * case["rot"]}
    if case["op"] == "decode":
        seen = sum(_visible(case, n) for n in _lengths(case))
        return {"bytes": seen * H * D * 4 + case["n_req"] * H * G * (4 * D + 4), "flops": 4 * seen * H * G * D}
    q, s = _lengths(case)
    r = _ranges(case)
    pairs = sum(a * b for a, b in zip(q, s)) if r is None else sum(e - b for b, e in r)
    return {"bytes": sum(s) * H * D * 4 + sum(q) * H * G * (4 * D + 4), "flops": 4 * pairs * H * G * D}


# ----------------------------------------------------------------- prepare
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _pages_for(lens, max_pages, slots, gen):
    """A page table over a random placement (unused entries -1)."""
    perm = torch.randperm(slots, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        p = -(-n // PAGE)
        table[b, :p] = perm[at:at + p]
        at += p
    return table, perm[at:]


def _pool(slots, H, D, gen, dtype):
    pool = torch.empty(slots, H, PAGE, D, dtype=dtype, device=DEV)
    for i in range(0, slots, 4096):  # in parts: no 32-bit copy of a whole pool
        pool[i:i + 4096] = torch.randn(pool[i:i + 4096].shape, device=DEV, generator=gen).to(dtype)
    return pool


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if own:
        import tiered_paged_kv_gb300 as tpk
        s["tpk"] = tpk
        code = tpk.BF16 if case.get("dtype") == "bf16" else tpk.F16
    if case["op"] == "tables":
        old, new = _lengths(case)
        used = sum(-(-n // PAGE) for n in old)
        want = sum(max(0, -(-b // PAGE) + (-a // PAGE)) for a, b in zip(old, new))
        free = int(want * (1 - case["short"])) + (64 if not case["short"] else 0)
        cap = used + free
        s["table"], rest = _pages_for(old, case["max_pages"], cap, gen)
        s["free"] = torch.full((cap,), -1, dtype=torch.int32, device=DEV)
        s["free"][:free] = rest
        s["n_free"], s["old"], s["new"] = _i32([free]), _i32(old), _i32(new)
        n = case["n_req"]
        s["max_tokens"] = sum(max(0, b - a) for a, b in zip(old, new)) + 37
        for k, (size, t) in {"n_free_out": (1, torch.int32), "len_out": (n, torch.int32), "granted": (n, torch.int32),
                             "tok_off": (n + 1, torch.int32), "slot_map": (s["max_tokens"], torch.int64),
                             "positions": (s["max_tokens"], torch.int32), "token_req": (s["max_tokens"], torch.int32)}.items():
            s[k] = torch.zeros(size, dtype=t, device=DEV)
        return s
    H, G, D, dt = case["H"], case["G"], case["D"], _dtype(case)
    rnd = lambda *shape: torch.randn(*shape, device=DEV, generator=gen).to(dt)  # noqa: E731
    if case["op"] == "rope":
        T, rot = case["tokens"], case["rot"]
        s["qkv"] = rnd(T, (H * G + 2 * H) * D)  # one projection's output: q, k and v side by side
        s["q"], s["k"], s["v"] = s["qkv"][:, :H * G * D], s["qkv"][:, H * G * D:(H * G + H) * D], s["qkv"][:, (H * G + H) * D:]
        slots = -(-T // PAGE) + 2
        s["k_pool"], s["v_pool"] = _pool(slots, H, D, gen, dt), _pool(slots, H, D, gen, dt)
        perm = torch.randperm(slots, device=DEV, generator=gen)
        i = torch.arange(T, device=DEV)
        s["slot_map"] = perm[i // PAGE] * PAGE + i % PAGE
        live = T - min(case["pad"], T - 1)
        s["slot_map"][live:] = -1  # padding rows of the batch
        s["live"] = live
        s["q_out"] = torch.zeros(T, H * G, D, dtype=dt, device=DEV)
        if case["axes"] == 1:
            s["positions"] = (torch.randint(0, case["far"], (1,), device=DEV, generator=gen) + i)[None].to(torch.int32)
            s["axis_of"] = np.zeros(rot // 2, np.uint8)
        else:  # frames of 24 x 32 patches; the frequencies go round the axes, the last ones all to time
            start = torch.randint(0, case["far"], (1,), device=DEV, generator=gen)
            s["positions"] = torch.stack([start + i // 768, start + i // 32 % 24, start + i % 32]).to(torch.int32)
            a = np.arange(rot // 2) % 3
            a[rot // 2 * 15 // 16:] = 0
            s["axis_of"] = a.astype(np.uint8)
        s["positions"] = s["positions"].contiguous()
        s["inv_freq"] = torch.tensor([1e6 ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float32, device=DEV)
        s["axis_dev"] = torch.tensor(s["axis_of"].astype(np.int64), device=DEV)
        if own:
            s["shape"] = tpk.PagedShape(H, G, D, dtype=code, kv_slots=slots)
        return s
    if case["op"] == "decode":
        lens = _lengths(case)
        s["q"] = rnd(case["n_req"], H * G, D)
        s["begin_host"] = [n - _visible(case, n) for n in lens]
        s["begin"] = _i32(s["begin_host"]) if case["window"] else None
        rows = case["n_req"]
    else:
        nq, lens = _lengths(case)
        s["nq"] = nq
        s["off"] = [sum(nq[:i]) for i in range(len(nq) + 1)]
        s["q_off"] = _i32(s["off"])
        s["q"] = rnd(sum(nq), H * G, D)
        r = _ranges(case)
        s["range"] = None if r is None else _i32(r)
        rows = sum(nq)
    s["lens_host"] = lens
    s["lens"] = _i32(lens)
    pages = sum(-(-n // PAGE) for n in lens)
    slots = pages + pages // 8 + 1
    max_pages = max(1, max(-(-n // PAGE) for n in lens))
    s["table"], _ = _pages_for(lens, max_pages, slots, gen)
    s["k_pool"], s["v_pool"] = _pool(slots, H, D, gen, dt), _pool(slots, H, D, gen, dt)
    s["o"] = torch.zeros(rows, H * G, D, dtype=dt, device=DEV)
    s["lse"] = torch.zeros(rows, H * G, dtype=torch.float32, device=DEV)
    if own:
        s["shape"] = tpk.PagedShape(H, G, D, dtype=code, kv_slots=slots, max_pages=max_pages)
        s["ws_bytes"] = (tpk.decode_paged_workspace_bytes(s["shape"], rows) if case["op"] == "decode"
                         else tpk.cross_paged_workspace_bytes(s["shape"], case["n_req"], rows))
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _plain_tables(s):
    old, new, mt, mp = s["old"].long(), s["new"].long(), s["max_tokens"], s["table"].shape[1]
    n = old.numel()
    grow = (new - old).clamp(min=0)
    off = torch.cat([grow.new_zeros(1), grow.cumsum(0)]).clamp(max=mt)
    have, want = -(-old // PAGE), -(-new // PAGE)
    fits = (want <= mp) & (off[:-1] + grow <= mt)
    take = torch.where(fits, (want - have).clamp(min=0), 0)
    give = torch.where(fits, (have - want).clamp(min=0), 0)
    n_free = s["n_free"].long()
    gave = give.cumsum(0)
    there = n_free + gave[-1:]
    taken = take.cumsum(0)
    granted = fits & ((take == 0) | (taken <= there))
    taken_all = torch.where(granted, taken, 0).max()
    n_free_out = there - taken_all
    # the stack after the releases: the free slots, then the pages given back
    j = torch.arange(mp, device=DEV)
    stack = torch.cat([s["free"], s["free"].new_zeros(n * mp)])
    back = (j >= want[:, None]) & (j < have[:, None]) & fits[:, None]
    at = n_free + (gave - give)[:, None] + j - want[:, None]
    stack = stack.scatter(0, torch.where(back, at, stack.numel() - 1).reshape(-1),
                          torch.where(back, s["table"], 0).reshape(-1))
    new_page = (j >= have[:, None]) & (j < want[:, None]) & granted[:, None]
    at = there - 1 - ((taken - take)[:, None] + j - have[:, None])
    table = torch.where(new_page, stack[torch.where(new_page, at, 0)], s["table"])
    k = torch.arange(s["free"].numel(), device=DEV)
    free = torch.where((k >= n_free) & (k < n_free_out), stack[:k.numel()], s["free"])
    t = torch.arange(mt, device=DEV)
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    real = b < n
    b = b.clamp(max=n - 1)
    pos = old[b] + t - off[b]
    ok = real & granted[b]
    page = torch.where(ok, pos // PAGE, 0)
    slot_map = torch.where(ok, table[b, page].long() * PAGE + pos % PAGE, -1)
    i32 = torch.int32
    return (table, free, n_free_out.to(i32), torch.where(granted, new, old).to(i32), granted.to(i32), off.to(i32), slot_map,
            torch.where(real, pos, 0).to(i32), torch.where(real, b, -1).to(i32))


def _own_tables(s):
    s["tpk"].kv_tables_update(s["case"]["n_req"], s["table"].shape[1], s["old"], s["new"], s["table"], s["free"],
                              s["free"].numel(), s["n_free"], s["n_free_out"], s["len_out"], s["granted"], s["tok_off"],
                              s["slot_map"], s["positions"], s["token_req"], s["max_tokens"],
                              stream=torch.cuda.current_stream())
    return (s["table"], s["free"], s["n_free_out"], s["len_out"], s["granted"], s["tok_off"], s["slot_map"], s["positions"],
            s["token_req"])


def _plain_rope(s):
    c = s["case"]
    H, G, D, rot, n = c["H"], c["G"], c["D"], c["rot"], s["live"]
    # far positions: the angle in 64 bits, its sine and cosine rounded to 32
    angle = s["positions"].double()[s["axis_dev"], :n].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x, heads):
        x = x[:n].float().view(n, heads, D)
        y = x.clone()
        if c["pairs"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(s["q"].dtype)

    s["q_out"][:n] = turn(s["q"], H * G)
    slot, row = s["slot_map"][:n] // PAGE, s["slot_map"][:n] % PAGE
    s["k_pool"][slot, :, row] = turn(s["k"], H)
    s["v_pool"][slot, :, row] = s["v"][:n].view(n, H, D)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_rope(s):
    c = s["case"]
    w = s["qkv"].stride(0)
    s["tpk"].kv_rope_append(s["shape"], c["tokens"], s["q"], w, s["k"], w, s["v"], w, s["positions"], c["axes"],
                            s["axis_of"], s["inv_freq"], c["rot"], c["pairs"], s["slot_map"], s["q_out"],
                            s["q_out"].stride(0), s["k_pool"], s["v_pool"], stream=torch.cuda.current_stream())
    return s["q_out"], s["k_pool"], s["v_pool"]


def _history(s, b, n, begin=0):
    """Request b's keys and values [begin, n) as [H, n - begin, D] in 32 bits."""
    first = begin // PAGE
    slots = s["table"][b, first:-(-n // PAGE)].long()
    out = []
    for pool in (s["k_pool"], s["v_pool"]):
        x = pool[slots].float().transpose(0, 1)
        out.append(x.reshape(x.shape[0], -1, x.shape[-1])[:, begin - first * PAGE:n - first * PAGE])
    return out


def _softmax(scores, v):
    """(softmax(scores) v, log of the sum); a row that sees nothing gives (0, -inf)."""
    m = scores.amax(-1, keepdim=True)
    safe = torch.where(m == NINF, 0.0, m)
    p = (scores - safe).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    return o, (safe + total.log())[..., 0]


def _plain_decode(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    for b, n in enumerate(s["lens_host"]):
        if n == s["begin_host"][b]:
            s["o"][b], s["lse"][b] = 0, NINF
            continue
        k, v = _history(s, b, n, s["begin_host"][b])
        scores = (s["q"][b].float().view(H, G, D) @ k.transpose(1, 2)) * D ** -0.5
        o, lse = _softmax(scores, v)
        s["o"][b], s["lse"][b] = o.reshape(H * G, D), lse.reshape(-1)
    return s["o"], s["lse"]


def _own_decode(s):
    w = s["q"].stride(0)
    s["tpk"].decode_attn_paged(s["shape"], s["case"]["n_req"], s["q"], w, s["k_pool"], s["v_pool"], s["table"], s["lens"],
                               s["begin"], s["o"], w, False, s["lse"], s["ws"], s["ws_bytes"],
                               stream=torch.cuda.current_stream())
    return s["o"], s["lse"]


def _plain_cross(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    for b, n in enumerate(s["lens_host"]):
        k, v = _history(s, b, n)
        i, e = s["off"][b], s["off"][b + 1]
        hide = None
        if s["range"] is not None:
            at = torch.arange(n, device=DEV)
            r = s["range"][i:e, :, None]
            hide = ((at < r[:, 0]) | (at >= r[:, 1]))[:, None]
        for h in range(H):
            q = s["q"][i:e, h * G:(h + 1) * G].float()
            scores = (q @ k[h].T) * D ** -0.5
            if hide is not None:
                scores = scores.masked_fill(hide, NINF)
            s["o"][i:e, h * G:(h + 1) * G], s["lse"][i:e, h * G:(h + 1) * G] = _softmax(scores, v[h])
    return s["o"], s["lse"]


def _own_cross(s):
    w = s["q"].stride(0)
    s["tpk"].cross_attn_paged(s["shape"], s["case"]["n_req"], s["q"].shape[0], s["q"], w, s["q_off"], s["k_pool"], s["v_pool"],
                              s["table"], s["lens"], s["range"], s["o"], w, s["lse"], s["ws"], s["ws_bytes"],
                              stream=torch.cuda.current_stream())
    return s["o"], s["lse"]


_run_plain = {"tables": _plain_tables, "rope": _plain_rope, "decode": _plain_decode, "cross": _plain_cross}
_run_own = {"tables": _own_tables, "rope": _own_rope, "decode": _own_decode, "cross": _own_cross}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "decode": _exact_attention, "cross": _exact_attention}[case["op"]](s)


def _exact_tables(s):
    """The same by a free stack and a loop over the requests."""
    old, new, mt = s["old"].tolist(), s["new"].tolist(), s["max_tokens"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    mp, n_free = table.shape[1], int(s["n_free"])
    pages = lambda x: (x + PAGE - 1) // PAGE  # noqa: E731
    off = [0]
    for a, b in zip(old, new):
        off.append(min(mt, off[-1] + max(0, b - a)))
    fits = [pages(b) <= mp and off[i] + max(0, b - a) <= mt for i, (a, b) in enumerate(zip(old, new))]
    stack = free[:n_free].tolist()
    for i, (a, b) in enumerate(zip(old, new)):
        if fits[i]:
            stack += table[i, pages(b):pages(a)].tolist()
    granted, length, full = [], [], False
    for i, (a, b) in enumerate(zip(old, new)):
        need = max(0, pages(b) - pages(a)) if fits[i] else 0
        full = full or need > len(stack)
        ok = fits[i] and (need == 0 or not full)
        for p in range(need if ok else 0):
            table[i, pages(a) + p] = stack.pop()
        granted.append(int(ok))
        length.append(b if ok else a)
    if len(stack) > n_free:
        free[n_free:len(stack)] = stack[n_free:]
    slot, pos, req = np.full(mt, -1, np.int64), np.zeros(mt, np.int32), np.full(mt, -1, np.int32)
    for i in range(len(old)):
        for t in range(off[i], off[i + 1]):
            p = old[i] + t - off[i]
            pos[t], req[t] = p, i
            if granted[i]:
                slot[t] = int(table[i, p // PAGE]) * PAGE + p % PAGE
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    return table, free, i32([len(stack)]), i32(length), i32(granted), i32(off), slot, pos, req


def _exact_rope(s):
    c = s["case"]
    n, rot, D = s["live"], c["rot"], c["D"]
    pos = s["positions"].double()
    out = []
    for x, heads in ((s["q"], c["H"] * c["G"]), (s["k"], c["H"])):
        x = x[:n].double().reshape(n, heads, D)
        y = x.clone()
        for j in range(rot // 2):
            lo, hi = (2 * j, 2 * j + 1) if c["pairs"] else (j, j + rot // 2)
            turn = torch.polar(torch.ones_like(pos[0, :n]), pos[int(s["axis_of"][j]), :n] * float(s["inv_freq"][j]))
            z = torch.complex(x[:, :, lo], x[:, :, hi]) * turn[:, None]
            y[:, :, lo], y[:, :, hi] = z.real, z.imag
        out.append(y)
    q_out, kp, vp = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
    q_out[:n] = out[0]
    where = s["slot_map"][:n].tolist()
    at = torch.tensor([w // PAGE * c["H"] * PAGE + h * PAGE + w % PAGE for w in where for h in range(c["H"])], device=DEV)
    kp.view(-1, D)[at] = out[1].reshape(-1, D)
    vp.view(-1, D)[at] = s["v"][:n].double().reshape(-1, D)
    return q_out, kp, vp


def _exact_attention(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    o, lse = s["o"].double(), s["lse"].double()
    for b, n in enumerate(s["lens_host"]):
        rows = slice(b, b + 1) if c["op"] == "decode" else slice(s["off"][b], s["off"][b + 1])
        q = s["q"][rows].double()
        seen = torch.ones(q.shape[0], n, dtype=torch.bool, device=DEV)
        at = torch.arange(n, device=DEV)
        if c["op"] == "decode":
            seen &= at >= s["begin_host"][b]
        elif s["range"] is not None:
            seen &= (at >= s["range"][rows, :1]) & (at < s["range"][rows, 1:])
        page = s["table"][b].long().repeat_interleave(PAGE)[:n]
        bias = torch.zeros(seen.shape, dtype=torch.float64, device=DEV).masked_fill(~seen, NINF)
        for j in range(H * G):
            k = s["k_pool"][page, j // G, at % PAGE].double()
            logits = torch.einsum("td,nd->tn", q[:, j], k) / D ** 0.5 + bias
            total = torch.logsumexp(logits, 1) if n else torch.full((q.shape[0],), NINF, dtype=torch.float64, device=DEV)
            weight = torch.where(seen, (logits - total[:, None]).exp(), 0.0)
            lse[rows, j] = total
            o[rows, j] = torch.einsum("tn,nd->td", weight, s["v_pool"][page, j // G, at % PAGE].double())
    return o, lse
