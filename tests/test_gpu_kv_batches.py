"""Batches of the 8-bit cache calls that hold less, or other, than their sizes let one expect: rows that no
sequence has, and index arrays that make no sense (reported, and never followed).  Bars as in test_gpu_kv."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_kv import Setup, bf, check_attend, i32  # noqa: E402


@pytest.mark.parametrize("group", [1, 4, 16, 20])
@pytest.mark.parametrize("q_len,max_q,rows", [(1, 1, 8), (1, 1, 40), (3, 4, 9), (5, 5, 300), (0, 1, 8), (40, 60, 64)])
def test_one_sequence_in_a_longer_step(qlin, group, q_len, max_q, rows):
    """One sequence whose step has rows behind it that are not in use: its rows, on both sides of the limit
    between the kernels, are right, and the others are left alone."""
    H, D = 2, 64
    su = Setup(qlin, "int8", D, 32, H, [q_len], [150], seed=group)
    q = su.rows(H * group, T=rows)
    b = qlin.KVBatch(i32([0, q_len]), i32([150]), i32(su.pages), rows, max_q, 150)
    o = torch.full((rows, H * group, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, H * group), 77.0, device="cuda")
    su.cache.attend(b, bf(q), out=o, lse=lse)
    su.ok()
    check_attend(su, q[:q_len], H * group, o[:q_len], lse[:q_len], D ** -0.5)
    assert bool((o[q_len:] == 77).all()) and bool((lse[q_len:] == 77).all())


@pytest.mark.parametrize("group", [1, 4, 20])
@pytest.mark.parametrize("n,max_q,rows", [(8, 1, 8), (30, 4, 30), (300, 5, 300)])
def test_one_sequence_with_more_tokens_than_said(qlin, group, n, max_q, rows):
    su = Setup(qlin, "int8", 64, 32, 2, [n], [400])
    q = bf(su.rows(2 * group))
    su.cache.attend(qlin.KVBatch(i32([0, n]), i32([400]), i32(su.pages), rows, max_q, 400), q)
    assert su.cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG


BIG = 2 ** 31


@pytest.mark.parametrize("q_start", [(BIG - 1, -BIG), (BIG - 3, -BIG + 1), (-BIG, BIG - 1), (-1, 0), (-1, 1), (0, BIG - 1), (1, 0),
                                     (3, 5), (4, 5), (5, 5)])
@pytest.mark.parametrize("group,max_q", [(2, 4), (20, 4)])
def test_q_start_out_of_range(qlin, q_start, group, max_q):
    """Sequences that are not rows 0..4 of the step, differences that wrap 32 bits among them."""
    su = Setup(qlin, "int8", 64, 16, 1, [4], [40])
    b = qlin.KVBatch(i32(q_start), i32([40]), i32(su.pages), 4, max_q, 40)
    x = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((4, group, 64), dtype=torch.bfloat16, device="cuda")
    before = su.codes.clone()
    for call in (lambda: su.cache.append(b, x, x, q=q), lambda: su.cache.read(b), lambda: su.cache.attend(b, q)):
        call()
        assert su.cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    assert torch.equal(before, su.codes)


@pytest.mark.parametrize("q_start,total,kv_lens,group", [
    ((0, 2000, 300, 1500), 2000, (2000, 9000, 4000), 1),  # a search and a walk find different sequences
    ((0, 2000, 300, 1500), 2000, (2000, 400, 9000), 4),
    ((0, 40, 20, 60, 10, 100), 100, (40, 50, 60, 70, 200), 8),
    ((5, 3, 1, 0), 8, (10, 20, 30), 1),
    ((0, 8, 4, 8, 4, 8, 4, 8), 8, (9, 9, 9, 9, 9, 9, 9), 2),
    (tuple(range(64)) + (0,), 64, (20,) * 64, 2),         # the last of many falls
    (tuple(range(0, 4000, 10)) + (3000, 4000), 4000, (300,) * 401, 3),
])
@pytest.mark.parametrize("q", [True, False])
def test_decreasing_q_start_is_reported(qlin, q_start, total, kv_lens, group, q):
    """A q_start that falls is reported as a bad index by every call, which then makes no access that it
    should not and does not hang; the workspace is good for the next call."""
    D, page, n = 64, 64, len(kv_lens)
    pages = -(-max(kv_lens) // page)
    rng = torch.Generator(device="cuda").manual_seed(total)
    codes = torch.randint(0, 256, (pages, 1, 2, page * D), generator=rng, device="cuda", dtype=torch.uint8)
    cache = qlin.KVCache(codes, torch.rand((pages, 1, page // 16, 2), generator=rng, device="cuda") * 0.01)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(n, pages).contiguous()
    b = qlin.KVBatch(i32(q_start), i32(kv_lens), table, total, total, max(kv_lens))
    x = torch.randn((total, 1, D), generator=rng, device="cuda").to(torch.bfloat16)
    one = qlin.KVBatch(i32(q_start), i32(kv_lens), table, total, 1, max(kv_lens))  # said to have single tokens
    y = torch.randn((total, group, D), generator=rng, device="cuda").to(torch.bfloat16)
    good = qlin.KVBatch(i32([0, total]), i32([max(kv_lens)]), table[:1], total, total, max(kv_lens))
    want = cache.attend(good, y)
    assert cache.poll_status() == 0
    cache.read(b)
    assert cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    cache.attend(b, y)
    assert cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    assert torch.equal(cache.attend(good, y), want)
    cache.append(b, x, x, q=y if q else None)
    assert cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    for call in (lambda: cache.read(one), lambda: cache.attend(one, y), lambda: cache.append(one, x, x, q=y if q else None)):
        call()
        assert cache.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    cache.append(good, x, x)
    assert cache.poll_status() == 0


def test_errors_outlive_a_cache_on_the_same_workspace(qlin):
    """A bad index that nobody has polled for is still there after another layer's cache took the workspace."""
    su = Setup(qlin, "int8", 64, 16, 1, [1], [40])
    pages = su.pages.copy()
    pages[0, 2] = -5
    q = bf(su.rows(2))
    su.cache.attend(su.make_batch([1], pages=pages), q)
    second = qlin.KVCache(su.codes.clone(), su.scales.clone(), workspace=su.cache.workspace)
    assert second.poll_status() == qlin.QLIN_ERR_INVALID_ARG
    assert torch.equal(second.attend(su.batch, q), su.cache.attend(su.batch, q))
    su.ok()


def pool_of(x):
    """The stream whose pool a tensor's memory comes from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= x.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_outputs_belong_to_the_stream_of_the_call(qlin):
    """Memory of the current stream's pool may still be in use by kernels queued there, which the stream of
    the call does not wait for: what a call on another stream makes comes from that stream's pool."""
    s = torch.cuda.Stream()
    su = Setup(qlin, "int8", 64, 16, 2, [3], [40])
    k, v, q = bf(su.rows(2)), bf(su.rows(2)), bf(su.rows(4))
    torch.cuda.synchronize()
    for given in (s, s.cuda_stream):
        qr = su.cache.append(su.batch, k, v, q=q, stream=given)
        o, lse = su.cache.attend(su.batch, qr, return_lse=True, stream=given)
        made = [qr, o, lse, *su.cache.read(su.batch, stream=given)]
        cache = qlin.KVCache.empty(4, 2, 64, 16, stream=given)
        made += [cache.codes, cache.scales, cache.workspace.memory]
        s.synchronize()
        assert [pool_of(x) for x in made] == [s.cuda_stream] * len(made)
    here = su.cache.attend(su.batch, qr)
    torch.cuda.synchronize()
    assert pool_of(here) == torch.cuda.current_stream().cuda_stream and torch.equal(here, o)
