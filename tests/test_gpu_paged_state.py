"""The state that PagedBatch carries from step to step: refused requests lose nothing, every page is in one
place, on any stream and in a graph."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from speculative_decoding_verify_06_gb300 import paged, svd
from tests.gpu_helpers import DEV, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def batch(R, **kw):
    a = dict(layers=1, n_pages=8, page_size=16, max_len=64, max_window=64, n_q_heads=2, n_kv_heads=1)
    return paged.PagedBatch(R, **{**a, **kw})


def whole(b):
    """Every page is held by one request or free."""
    held, table = b.held[b.now].tolist(), b.table[b.now].cpu().numpy()
    have = [-(-h // b.page) for h in held]
    ids = np.concatenate([table[r, :n] for r, n in enumerate(have)] + [b.free[b.now].cpu().numpy()[:int(b.n_free[b.now])]])
    assert np.array_equal(np.sort(ids), np.arange(b.n_pages))
    assert all((table[r, n:] == -1).all() for r, n in enumerate(have))


def test_carried_state_against_the_definitions():
    """Whole outputs of the call, over random states and counts in and out of order."""
    g = np.random.default_rng(7)
    for R, page, width, spare, tokens in ((1, 16, 3, 2, 40), (37, 32, 6, 9, 150), (700, 16, 4, 200, 3000)):
        held = g.integers(0, width * page + 1, R)
        have = -(-held // page)
        ids = g.permutation(int(have.sum()) + spare).astype(np.int32)
        table = np.full((R, width), -1, np.int32)
        table[np.arange(width) < have[:, None]] = ids[:have.sum()]
        free = np.full(len(ids), -1, np.int32)
        free[:spare] = ids[have.sum():]
        window = np.minimum(held, g.integers(0, 12, R)) * g.choice([1, 1, -1], R)
        window[g.random(R) < 0.1] += 1000
        emitted = np.maximum(window, 0) - g.integers(-1, 4, R)
        n_new = g.integers(-1, 20, R)
        for kept, most in ((emitted, 15), (None, 1 << 20), (emitted, 2)):
            want = ref.advance(held, window, kept, n_new, most, page, table, free, spare, tokens)
            d = {k: torch.full(np.shape(v) or (1,), -77, dtype=torch.int64 if k == "slots" else torch.int32, device=DEV)
                 for k, v in want.items()}
            ins = [None if a is None else i32(*a.reshape(-1).tolist()) for a in (held, window, kept, n_new, table, free)]
            svd.svd_paged_advance(*ins[:4], R, most, page, ins[4], width, ins[5], i32(spare), len(ids), d["held"], d["window"],
                                  d["table"], d["free"], d["n_free"], d["kv_len"], d["q_start"], d["slots"], d["positions"],
                                  tokens, d["status"])
            for k in want:
                assert np.array_equal(d[k].cpu().numpy().reshape(np.shape(want[k])), want[k]), k


def test_a_request_that_reaches_its_longest_keeps_its_cache():
    b = batch(2)
    b.begin(i32(60, 3))
    row = b.table[b.now][0].tolist()
    b.begin(i32(8, 2), i32(60, 3))  # 68 positions do not fit
    assert b.status.tolist() == [svd.SVD_ST_BAD_REQUEST, 0] and b.q_start.tolist() == [0, 0, 2]
    whole(b)
    assert b.table[b.now][0].tolist() == row
    for kept in (i32(0, 1), i32(5, 1)):  # counts of a request that had no tokens say nothing
        b.begin(i32(8, 2), kept)
        assert b.status.tolist() == [svd.SVD_ST_BAD_REQUEST, 0]
        whole(b)
    b.begin(i32(4, 0))
    assert b.status.tolist() == [0, 0] and b.kv_len.tolist()[0] == 64 and b.positions[:4].tolist() == [60, 61, 62, 63]
    assert b.table[b.now][0].tolist() == row
    whole(b)


def test_a_request_refused_for_pages_after_rejected_drafts():
    b = batch(2, n_pages=4)
    b.begin(i32(30, 10))
    b.begin(i32(10, 0), i32(30, 10))  # request 0 holds 40: three pages; none is left
    assert b.kv_len.tolist() == [40, 10] and int(b.n_free[b.now]) == 0
    b.begin(i32(33, 0), i32(1, 0))    # of ten drafts one stays: 31, and 64 do not fit
    assert b.status.tolist() == [svd.SVD_ST_NO_PAGES, 0] and b.kv_len.tolist() == [31, 10]
    whole(b)
    b.begin(i32(33, 0), i32(9, 3))    # refused again; the count was settled with the first refusal
    assert b.status.tolist() == [svd.SVD_ST_NO_PAGES, 0] and b.kv_len.tolist() == [31, 10]
    whole(b)
    b.begin(i32(1, 0))                # 32 need two pages: the third goes back
    assert b.status.tolist() == [0, 0] and b.kv_len.tolist() == [32, 10] and b.positions[0].item() == 31
    assert int(b.n_free[b.now]) == 1
    whole(b)


def test_a_request_refused_for_tokens_after_rejected_drafts():
    b = batch(2, max_tokens=20)
    b.begin(i32(16, 4))
    b.begin(i32(4, 16), i32(14, 4))
    assert b.kv_len.tolist() == [18, 20]
    b.begin(i32(10, 11), i32(1, 2))
    assert b.status.tolist() == [0, svd.SVD_ST_NO_TOKENS] and b.kv_len.tolist() == [25, 6]
    whole(b)
    b.begin(i32(0, 1))
    assert b.status.tolist() == [0, 0] and b.kv_len.tolist() == [25, 7] and b.positions[0].item() == 6
    whole(b)


def test_counts_out_of_order_are_asked_for_again():
    b = batch(1)
    b.begin(i32(20))
    for bad in (i32(21), i32(-1)):
        b.begin(i32(2), bad)
        assert b.status.tolist() == [svd.SVD_ST_BAD_REQUEST]
        whole(b)
    b.begin(i32(2), i32(17))
    assert b.status.tolist() == [0] and b.kv_len.tolist() == [19] and b.positions[:2].tolist() == [17, 18]
    whole(b)


@pytest.mark.parametrize("seed", range(4))
def test_many_steps_against_the_definitions(seed):
    """Refusals of every kind, again and again, beside a list of the positions each request should hold."""
    g = np.random.default_rng(seed)
    R, page, n_pages, longest, tokens = 6, 16, 14, 80, 60
    b = batch(R, n_pages=n_pages, max_len=longest, max_tokens=tokens, max_window=longest)
    kept, last, seen = [0] * R, [0] * R, set()  # positions kept before the last window; the last window
    for step in range(80):
        emitted = [int(g.integers(0, w + 1)) if w else int(g.integers(0, 5)) for w in last]
        wrong = g.random(R) < 0.05
        given = [w + 1 if x and w else e for e, w, x in zip(emitted, last, wrong)]
        n = [int(g.choice([0, 1, 4, 9, 30])) if g.random() < 0.97 else -1 for _ in range(R)]
        b.begin(i32(*n), i32(*given))
        status = b.status.tolist()
        seen |= set(status)
        for r in range(R):
            if wrong[r] and last[r]:
                assert status[r] == svd.SVD_ST_BAD_REQUEST
                continue  # the window waits for its count
            kept[r] += emitted[r] if last[r] else 0
            last[r] = n[r] if status[r] == 0 else 0
            assert (status[r] == svd.SVD_ST_BAD_REQUEST) == (n[r] < 0 or kept[r] + n[r] > longest)
            assert b.kv_len.tolist()[r] == kept[r] + last[r]
        granted = [n[r] if status[r] == 0 else 0 for r in range(R)]
        assert b.q_start.tolist() == np.concatenate([[0], np.cumsum(granted)]).tolist()
        table, pos, slots = b.table[b.now].cpu().numpy(), b.positions.tolist(), b.slots.tolist()
        t = 0
        for r in range(R):
            for i in range(granted[r]):
                assert pos[t] == kept[r] + i and slots[t] == table[r, pos[t] // page] * page + pos[t] % page
                t += 1
        whole(b)
        if step % 16 == 15:  # start some anew: what is held and not kept goes back
            b.begin(i32(*[0] * R), i32(*[0] * R))
            for r in range(R):
                if b.status.tolist()[r] == 0:
                    last[r] = 0
            whole(b)
    assert {0, svd.SVD_ST_BAD_REQUEST, svd.SVD_ST_NO_PAGES, svd.SVD_ST_NO_TOKENS} <= seen


def test_a_step_on_a_stream_that_is_not_the_current_one():
    s = torch.cuda.Stream()
    batch(2).begin(i32(1, 1), stream=s)  # (kernels are loaded at their first use, which waits for the device)
    b = batch(2)
    new, kept = [i32(10, 20), i32(3, 3), i32(2, 2)], [None, i32(4, 20), i32(1, 3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # the current stream is busy for a fifth of a second
    for n, k in zip(new, kept):
        b.begin(n, k, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(s):
        assert b.status.tolist() == [0, 0] and b.kv_len.tolist() == [7, 25] and b.window.tolist() == [2, 2]
    torch.cuda.synchronize()
    whole(b)


def test_more_tokens_than_a_window_holds_are_refused():
    """What the attention would leave without outputs gets no slots either; the rest is served."""
    b = batch(3, max_window=5, max_tokens=12)
    b.begin(i32(5, 6, 4))
    assert b.status.tolist() == [0, svd.SVD_ST_NO_TOKENS, 0]
    assert b.q_start.tolist() == [0, 5, 5, 9] and b.kv_len.tolist() == [5, 0, 4]
    b.max_window = 4
    b.begin(i32(5, 4, 4), i32(2, 3, 4))
    assert b.status.tolist() == [svd.SVD_ST_NO_TOKENS, 0, 0] and b.kv_len.tolist() == [2, 4, 8]
    whole(b)
    b.max_window = 1  # (for the next step)
    # every token with a slot has its output
    x = torch.randn((12, 4 * 128), device=DEV)
    out = torch.full((12, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    b.layer(0, x, out)
    assert torch.isfinite(out[:8]).all() and torch.isnan(out[8:]).all() and (b.slots[:8] >= 0).all() and (b.slots[8:] < 0).all()


@pytest.mark.parametrize("raw", [False, True])
def test_one_step_recorded_and_replayed(raw):
    """A graph of a single step goes on from where the last replay, or the last step outside it, ended."""
    R, n = 3, 2

    def make():
        b = paged.PagedBatch(R, 1, n_pages=40, page_size=16, max_len=256, max_window=n, n_q_heads=4, n_kv_heads=2,
                             rope=svd.Rope(np.full(64, 0.3)))
        g = torch.Generator(device=DEV)
        g.manual_seed(3)
        return (b, torch.randn((R * n, 8 * 128), generator=g, device=DEV),
                torch.zeros((R * n, 4, 128), dtype=torch.bfloat16, device=DEV), i32(1, 2, 1))

    new = i32(*[n] * R)
    b, x, out, kept = make()
    b.begin(new)
    want = []
    for step in range(7):
        b.begin(new, kept)
        b.layer(0, x, out)
        want.append((out.clone(), b.kv_len.tolist(), b.slots.tolist()))
    b, x, out, kept = make()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.begin(new)
    s.synchronize()

    def step(stream=None):
        b.begin(new, kept, stream=stream)
        b.layer(0, x, out, stream=stream)
    if raw:
        svd.svd_graph_begin(s)
        step(s.cuda_stream)
        graph = svd.svd_graph_end(s)
        play = lambda: graph.launch(s)  # noqa: E731
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        play = graph.replay
    with torch.cuda.stream(s):
        for i, (o, lens, slots) in enumerate(want):
            if i == 3:
                step()  # one outside the graph
            else:
                play()
            assert torch.equal(out, o) and b.kv_len.tolist() == lens and b.slots.tolist() == slots, i
    torch.cuda.synchronize()
    whole(b)


def test_a_request_that_ends_gives_its_pages_back():
    b = batch(3)
    b.begin(i32(40, 20, 33))
    b.end(torch.tensor([False, True, True], device=DEV))
    b.begin(i32(2, 0, 50), i32(39, 7, 5))  # request 2's place goes to another one at once
    assert b.status.tolist() == [0, 0, 0] and b.kv_len.tolist() == [41, 0, 50]
    assert b.positions[:52].tolist() == [39, 40] + list(range(50)) and int(b.n_free[b.now]) == 8 - 3 - 4
    whole(b)
    b.end(torch.tensor([True, False, False], device=DEV))
    b.begin(i32(4, 33, 64), i32(2, 0, 50))  # a refusal beside the end: request 2's length
    assert b.status.tolist() == [0, 0, svd.SVD_ST_BAD_REQUEST] and b.kv_len.tolist() == [4, 33, 50]
    b.end(torch.tensor([True, True, True], device=DEV))
    b.begin(i32(0, 65, 0))                  # an end holds through a refusal
    assert b.status.tolist() == [0, svd.SVD_ST_BAD_REQUEST, 0] and b.kv_len.tolist() == [0, 0, 0]
    whole(b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.begin(i32(0, 0, 0), i32(9, 9, 9), stream=s)
    s.synchronize()
    assert int(b.n_free[b.now]) == 8
    b.begin(i32(20, 20, 20), stream=s)
    b.end(torch.ones(3, dtype=torch.bool, device=DEV), stream=s)
    b.begin(i32(0, 0, 1), stream=s)
    s.synchronize()
    assert b.kv_len.tolist() == [0, 0, 1] and int(b.n_free[b.now]) == 7
    whole(b)


def test_a_wait_that_gave_up_is_seen():
    b = batch(1, max_window=40)
    b.begin(i32(40))
    x, out = torch.randn((40, 4 * 128), device=DEV), torch.zeros((40, 2, 128), dtype=torch.bfloat16, device=DEV)
    b.layer(0, x, out)
    assert b.attention_status.tolist() == [0]
    want = out.clone()
    b.ws[4:8].view(torch.int32).fill_(1)  # every wait that is not satisfied at once gives up
    b.layer(0, x, out)
    assert b.attention_status.tolist() == [1]
    b.ws[4:8] = 0
    b.layer(0, x, out)
    assert b.attention_status.tolist() == [1] and torch.equal(out, want)
    b.attention_status.zero_()
    assert b.attention_status.tolist() == [0]


@pytest.mark.parametrize("handle", ["stream", "address", "default"])
def test_streams_in_every_form(handle):
    busy = torch.cuda.Stream()
    s = torch.cuda.default_stream() if handle == "default" else torch.cuda.Stream()
    given = s if handle == "stream" else s.cuda_stream
    assert given == 0 or handle != "default"
    b, warm = batch(2), batch(2)
    new, who = i32(10, 20), torch.tensor([False, True], device=DEV)
    warm.begin(new, stream=given)
    warm.end(who, stream=given)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)  # what runs anywhere else comes too early
    with torch.cuda.stream(busy):
        torch.cuda._sleep(800_000_000)
        b.begin(new, stream=given)
        b.end(who, stream=given)
        b.begin(new, stream=given)
        s.synchronize()
        assert not busy.query()
        with torch.cuda.stream(s):
            assert b.kv_len.tolist() == [20, 20] and b.held[b.now].tolist() == [20, 20]
        assert not busy.query()
    torch.cuda.synchronize()
    whole(b)
