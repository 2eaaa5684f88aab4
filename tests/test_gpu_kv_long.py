"""Attention over the 8-bit cache on long contexts and big batches, against float64 in plain PyTorch
on the GPU (the numpy oracle of the other tests is too slow for these sizes).

Bars, derived before any run, term by term as in the tests of short contexts, but with the weights' range:
a row's fp16 weights are held with their largest at 2^10 or above, so a small one is off by at most 2^-25 of
2^-10 of the largest, which moves an output by up to 2^-35 max(p vs) sum|cv| (p: weights, vs, cv: scales and
codes of the values).  With a factor of 16 of room for that term and 2 for the others:
|o - o_ref| <= 2^-8 |o_ref| + (2^-10 + 2^-14 (1 + mag)) sum p|v| + 2^-31 max(p vs) sum|cv|,
|lse - ref| <= 2^-16 (1 + mag), mag = the row's largest scale * sum |q||k|.
"""
import numpy as np
import pytest

from oracle import kv as okv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Long:
    """One long sequence of T tokens in the cache (pages in a shuffled order), which the sequences of a
    batch share: sequence b is its first kv_lens[b] tokens."""

    def __init__(self, qlin, code, D, page, H, T, seed=0, keys=1.0, values=1.0, mean=0.0):
        self.qlin, self.code, self.D, self.page, self.H, self.T = qlin, code, D, page, H, T
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        n = -(-T // page)
        self.order = torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32)
        k = torch.randn(T, H, D, generator=g, device="cuda") * keys
        v = torch.randn(T, H, D, generator=g, device="cuda") * values + mean
        self.codes = torch.randint(0, 256, (n + 2, H, 2, page * D), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = torch.full((n + 2, H, page // 16, 2), float("nan"), device="cuda")
        self.cache = qlin.KVCache(self.codes, self.scales, code)
        self.store(k, v)

    def store(self, k, v):
        """Quantizes k, v [T, H, D] block by block, in plain PyTorch."""
        T, page, top = self.T, self.page, float(okv.QMAX[self.code])
        nb = page // 16
        for which, x in ((0, k), (1, v)):
            pad = torch.zeros((self.order.numel() * page, self.H, self.D), device="cuda")
            pad[:T] = x
            b = pad.view(-1, nb, 16, self.H, self.D).permute(0, 3, 1, 2, 4)  # page, head, block, token, element
            s = (b.abs().amax((3, 4)) / top).clamp_min(2.0 ** -60)
            y = b / s[..., None, None]
            if self.code == "int8":
                byte = (y.round().clamp(-127, 127) + 128).to(torch.uint8)
            else:
                byte = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            if which:
                byte = byte.transpose(3, 4)  # a block's tokens innermost
            at = self.order.long()
            self.codes[at, :, which] = byte.reshape(len(at), self.H, page * self.D)
            self.scales[at, :, :, which] = s

    def batch(self, q_lens, kv_lens):
        cols = max(-(-max(kv_lens) // self.page), 1)
        pages = self.order[:cols].expand(len(kv_lens), cols).contiguous()
        return self.qlin.KVBatch(i32(np.concatenate([[0], np.cumsum(q_lens)])), i32(kv_lens), pages, int(sum(q_lens)),
                                 max(q_lens), max(kv_lens))

    def held(self):
        """Codes and scales of the keys and values, [H, T, D] and [H, T, 1], float64."""
        nb, at, out = self.page // 16, self.order.long(), []
        for which in (0, 1):
            c = self.codes[at, :, which]
            c = c.double() - 128 if self.code == "int8" else c.view(torch.float8_e4m3fn).double()
            shape = (-1, self.H, nb, self.D, 16) if which else (-1, self.H, nb, 16, self.D)
            c = c.reshape(shape)
            if which:
                c = c.transpose(3, 4)
            c = c.permute(1, 0, 2, 3, 4).reshape(self.H, -1, self.D)[:, :self.T]
            s = self.scales[at][..., which].double().permute(1, 0, 2)[..., None].expand(-1, -1, -1, 16)
            out += [c, s.reshape(self.H, -1, 1)[:, :self.T]]
        return out

    def check(self, q_lens, kv_lens, q, o, lse, scale, rows=None, window=0, sinks=0, slack=0.0):
        """Compares the given rows (sequence, token), all by default."""
        kc, ks, vc, vs = self.held()
        hq = q.shape[1]
        group = hq // self.H
        starts = np.concatenate([[0], np.cumsum(q_lens)])
        worst = 0.0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            tokens = [t for t in range(n) if rows is None or (b, t) in rows]
            if not tokens:
                continue
            t = torch.tensor(tokens, device="cuda")
            pos = kv - n + t
            have = max(kv, 1)  # (a sequence of no tokens sees nothing of one)
            j = torch.arange(have, device="cuda")
            seen = j <= pos[:, None]
            if window:
                seen &= (j > pos[:, None] - window) | (j < sinks)
            for h in range(self.H):
                x = q[starts[b] + t, h * group:(h + 1) * group].double()  # [t, g, D]
                K, V = kc[h, :have] * ks[h, :have], vc[h, :have] * vs[h, :have]
                w = (x @ K.T * scale).masked_fill(~seen[:, None], -torch.inf)
                m = w.amax(-1, keepdim=True)
                none = torch.isneginf(m)
                p = torch.exp(w - torch.where(none, torch.zeros_like(m), m))
                total = p.sum(-1, keepdim=True)
                p = torch.where(none, torch.zeros_like(p), p / torch.where(none, torch.ones_like(total), total))
                ref = p @ V
                mag = ((x.abs() @ K.abs().T * scale) * seen[:, None]).amax(-1, keepdim=True)
                codes = seen.double() @ vc[h, :have].abs()
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -14 * (1 + mag)) * (p @ V.abs()) + \
                    2.0 ** -31 * (p * vs[h, :have, 0]).amax(-1, keepdim=True) * codes[:, None] + slack
                got = o[starts[b] + t, h * group:(h + 1) * group].double()
                assert bool(torch.isfinite(got).all())
                worst = max(worst, float(((got - ref).abs() / tol.clamp_min(1e-300)).max()))
                l = lse[starts[b] + t, h * group:(h + 1) * group, None].double()
                want = m + torch.log(total)
                assert bool((torch.isneginf(l) == none).all())
                assert bool((((l - want).abs() <= 2.0 ** -16 * (1 + mag)) | none).all())
        assert worst <= 1, f"worst {worst}"


def bf(x):
    return x.to(torch.bfloat16)


def some_rows(q_lens, n, seed):
    """n sequences, of each its first and last token and one between."""
    rng = np.random.default_rng(seed)
    live = [b for b, q in enumerate(q_lens) if q]
    pick = rng.choice(live, min(n, len(live)), replace=False)
    return {(int(b), int(t)) for b in pick for t in (0, q_lens[b] - 1, rng.integers(q_lens[b]))}


@pytest.mark.parametrize("code,D", [("int8", 64), ("e4m3", 128)])
@pytest.mark.parametrize("seqs,q_len,group", [(480, 1, 4), (480, 2, 8), (76, 16, 4), (38, 96, 4)])
def test_dominant_first_token(qlin, code, D, seqs, q_len, group):
    """A first token with 99.9% of the weight and a small value, before 32768 tokens whose values have a
    common mean: what they add up to is a tenth of the output.  So many sequences that a warp (a CTA, for
    prompts) has whole items, whose weights are held against the one large one all along."""
    T, H = 32768, 2
    su = Long(qlin, code, D, 64, H, T, seed=seqs, keys=0.02, mean=1.0, values=0.3)
    direction = torch.randn(H, D, generator=su.g, device="cuda")
    k = torch.randn(T, H, D, generator=su.g, device="cuda") * 0.02
    v = torch.randn(T, H, D, generator=su.g, device="cuda") * 0.3 + 1.0
    q = direction.repeat_interleave(group, 0) + 0.02 * torch.randn(seqs * q_len, H * group, D, generator=su.g, device="cuda")
    scale = D ** -0.5
    k[0] = direction * (np.log(999.0 * T) / (scale * (direction ** 2).sum(-1, keepdim=True)))
    v[0] = 0.01 * torch.randn(H, D, generator=su.g, device="cuda")
    su.store(k, v)
    q_lens, kv_lens = [q_len] * seqs, [T - b % 16 for b in range(seqs)]
    q = bf(q)
    o, lse = su.cache.attend(su.batch(q_lens, kv_lens), q, return_lse=True)
    assert su.cache.poll_status() == 0
    su.check(q_lens, kv_lens, q, o, lse, scale, some_rows(q_lens, 6, seqs))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,group", [([1, 1, 1], 4), ([2, 1, 3], 5), ([17, 40, 9], 3), ([200, 90, 30], 2)])
@pytest.mark.parametrize("which", ["values", "keys", "both", "all values", "tiny"])
def test_scales_of_zero(qlin, code, D, q_lens, group, which):
    """Blocks whose scale is 0, as an all-zero block of a cache from elsewhere may have it, with codes that
    are not 0: keys and values of 0, exactly."""
    T, H = 700, 2
    su = Long(qlin, code, D, 48, H, T, seed=D + len(which))
    some = torch.rand(su.scales.shape[:3], generator=su.g, device="cuda") < 0.4
    if which in ("values", "both"):
        su.scales[..., 1][some] = 0.0
    if which in ("keys", "both"):
        su.scales[..., 0][some.flip(0)] = 0.0
    if which == "all values":
        su.scales[..., 1] = 0.0
    if which == "tiny":  # under 2^-60, down to numbers without a reciprocal in fp32
        su.scales[..., 1][some] = torch.tensor([2.0 ** -61, 2.0 ** -100, 2.0 ** -140], device="cuda")[
            torch.randint(0, 3, (int(some.sum()),), generator=su.g, device="cuda")]
    kv_lens = [T, 333, 40]
    q = bf(torch.randn(sum(q_lens), H * group, D, generator=su.g, device="cuda"))
    o, lse = su.cache.attend(su.batch(q_lens, kv_lens), q, return_lse=True)
    assert su.cache.poll_status() == 0
    # (values of a scale under 2^-60 are themselves under 448 * 2^-60)
    su.check(q_lens, kv_lens, q, o, lse, D ** -0.5, slack=448 * 2.0 ** -60 if which == "tiny" else 0.0)
    if which == "all values":
        assert not bool(o.any())
    k, v = su.cache.read(su.batch([T], [T]))
    held = su.held()
    assert torch.equal(v.double(), (held[2] * held[3]).float().to(torch.bfloat16).double().transpose(0, 1))


# Work enough that every warp (CTA) goes round its rings and tables, takes several batches of lookups and
# several items, and joins them over all CTAs

def run(qlin, code, D, page, H, group, q_lens, kv_lens, window=0, sinks=0, seed=0, pick=None):
    su = Long(qlin, code, D, page, H, max(kv_lens), seed)
    q = bf(torch.randn(sum(q_lens), H * group, D, generator=su.g, device="cuda") * 1.5)
    batch = su.batch(q_lens, kv_lens)
    o, lse = su.cache.attend(batch, q, window=window, sinks=sinks, return_lse=True)
    assert su.cache.poll_status() == 0
    rows = None if pick is None else some_rows(q_lens, pick, seed)
    su.check(q_lens, kv_lens, q, o, lse, D ** -0.5, rows, window, sinks)
    again = su.cache.attend(batch, q, window=window, sinks=sinks)
    assert su.cache.poll_status() == 0 and torch.equal(o, again)


def lengths(seed, n, lo, hi):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi, n)]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2900, 20)])
def test_decode_many_units_a_warp(qlin, code, D, group, window, sinks):
    """64 sequences of 3000 to 5000 tokens, 8 heads: some 35 units of 64 tokens for each of 900 warps (rings of
    two or four stages, lookups of eight units), items that end anywhere in them."""
    run(qlin, code, D, 64, 8, group, [1] * 64, lengths(D + group, 64, 3000, 5000), window, sinks, seed=group, pick=24)


@pytest.mark.parametrize("code,D,group", [("int8", 128, 4), ("e4m3", 128, 16), ("int8", 64, 16), ("e4m3", 64, 1)])
def test_decode_item_over_all_ctas(qlin, code, D, group):
    """One head of one sequence of 210000 tokens: its parts are joined over all CTAs."""
    run(qlin, code, D, 128, 1, group, [1], [210007], seed=group)


@pytest.mark.parametrize("n", [193, 700, 2048])
@pytest.mark.parametrize("group,q_len", [(4, 1), (5, 3)])
def test_decode_many_sequences(qlin, n, group, q_len):
    """More sequences than a CTA has threads, up to the most: lengths from none on."""
    run(qlin, "int8", 64, 16, 2, group, [q_len] * n, lengths(n, n, 0, 300), seed=n, pick=200)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 20)])
@pytest.mark.parametrize("most", [30, 160])
def test_prompts_many_items_a_cta(qlin, code, D, window, sinks, most):
    """Up to 120 rows a head in every sequence (the variant for few rows), or up to 640 beside few: some five
    items and tens of key tiles a CTA, items of one and of two row tiles in turn."""
    n = 100 if most == 30 else 60
    q_lens = lengths(D, n, 5, most)
    kv_lens = [q + x for q, x in zip(q_lens, lengths(most, n, 500, 4500))]
    run(qlin, code, D, 48, 8, 4, q_lens, kv_lens, window, sinks, seed=most, pick=10)


@pytest.mark.parametrize("n,q_len,group", [(900, 20, 1), (2048, 40, 2), (2048, 9, 2)])
def test_prompts_many_row_blocks(qlin, n, q_len, group):
    """More row blocks than a CTA has threads."""
    q_lens = lengths(q_len, n, q_len - 3, q_len + 1)
    run(qlin, "int8", 64, 32, 1, group, q_lens, [max(q + x, 0) for q, x in zip(q_lens, lengths(n, n, -30, 400))],
        seed=q_len, pick=150)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_many_sequences(qlin, code):
    from test_gpu_kv import run_append
    n = 2048
    q = lengths(1, n, 0, 4)
    run_append(qlin, code, 64, 16, 1, q, [max(a + b, 0) for a, b in zip(q, lengths(2, n, -2, 20))], 64, hq=1)
    run_append(qlin, code, 64, 16, 1, [1] * n, lengths(3, n, 0, 20), 64, hq=1)


@pytest.mark.parametrize("qscale", [2.0 ** 16, 2.0 ** 20, 2.0 ** 23])
@pytest.mark.parametrize("q_lens,group", [([1, 1], 4), ([3, 4], 4), ([30, 9], 2), ([150, 40], 2)])
def test_scores_far_out(qlin, qscale, q_lens, group):
    """Scores so large that fp32 rounds them by whole powers of two of a weight: an output is one value or a
    mixture of a few, and stays among the values."""
    for code, D in (("int8", 64), ("e4m3", 128)):
        su = Long(qlin, code, D, 32, 2, 900, seed=D)
        q = bf(torch.randn(sum(q_lens), 2 * group, D, generator=su.g, device="cuda") * qscale)
        o = su.cache.attend(su.batch(q_lens, [900, 500]), q)
        assert su.cache.poll_status() == 0
        _, _, vc, vs = su.held()
        assert bool(torch.isfinite(o).all()) and float(o.abs().max()) <= float((vc * vs).abs().max()) * 1.01


@pytest.mark.parametrize("q_len", [1, 20])
def test_positions_past_2_30(qlin, q_len):
    """2^30 + 100 tokens in a table whose columns share two pages: a window over the whole table hides
    nothing, the first tokens among it, one of which has nearly all the weight."""
    D, page, T = 64, 1 << 20, (1 << 30) + 100
    su = Long(qlin, "int8", D, page, 1, 2 * page, seed=q_len, keys=0.02)
    x = torch.randn(D, generator=su.g, device="cuda")
    k = torch.randn(2 * page, 1, D, generator=su.g, device="cuda") * 0.02
    v = torch.randn(2 * page, 1, D, generator=su.g, device="cuda")
    k[5, 0] = x * 40 / (D ** -0.5 * (x * x).sum())
    su.store(k, v)
    table = su.order[1].expand(1, -(-T // page)).clone()
    table[0, 0] = su.order[0]
    batch = qlin.KVBatch(i32([0, q_len]), i32([T]), table, q_len, q_len, T)
    q = bf(x.expand(q_len, 1, D).contiguous())
    want, lse = su.cache.attend(batch, q, return_lse=True)
    _, _, vc, vs = su.held()
    value = (vc[0, 5] * vs[0, 5]).float()
    assert float((want.float() - value).abs().max()) < 0.02 and bool((lse > 38).all())
    for window, sinks in ((2 ** 31 - 1, 0), (page * table.shape[1], 0), (100, 2 ** 31 - 1), (2 ** 30, 6)):
        got, l = su.cache.attend(batch, q, window=window, sinks=sinks, return_lse=True)
        if window != 2 ** 30:  # (that one hides some of the first tokens, not the sixth)
            assert torch.equal(got, want) and torch.equal(l, lse)
        assert float((got.float() - value).abs().max()) < 0.02
    hidden, l = su.cache.attend(batch, q, window=2 ** 30, return_lse=True)
    assert float(l.max()) < 30
    assert su.cache.poll_status() == 0
