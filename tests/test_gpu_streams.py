"""The `stream` argument of the conveniences.  What a call allocates belongs to the stream
that it runs on: it must neither take memory that work of the current stream still uses, nor
give memory that it still uses itself to that stream.  The streams are held up by a kernel
that spins for a fixed number of cycles."""
import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

SPIN = 20_000_000  # 8 ms, far more than the host takes for a call


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def step_calls(svd):
    """(name, call(**kw) -> tuple of result tensors) of the calls around a step."""
    torch.manual_seed(5)
    B, T, Hq, Hkv, D, page, mp = 3, 9, 8, 2, 128, 16, 60
    c = svd.kv_cache(B * mp, Hkv, page, D)
    tab = torch.arange(B * mp, dtype=torch.int32, device="cuda").view(B, mp)
    ctx, start, hlen = i32(800, 17, 450), i32(1, 2, 3), i32(40, 3, 0)
    k = torch.randn(2, B, 900, Hkv, D, device="cuda", dtype=torch.bfloat16)
    svd.cache_write(c, k[0], k[1], tab, i32(0, 0, 0))
    q = torch.randn(B, T, Hq, D, device="cuda", dtype=torch.bfloat16)
    assert svd.tree_attention_workspace(B, T, Hq, c, tab).numel() > 256  # parts are joined
    drafts = torch.randint(0, 9, (B, 6, 7), dtype=torch.int32, device="cuda")
    z = torch.randn(B, T, 5003, device="cuda")
    h = torch.randint(0, 5003, (B, 40), dtype=torch.int32, device="cuda")
    f = torch.full((B,), 0.25, device="cuda")

    def tree(**kw):
        return tuple(svd.draft_tree(drafts, **kw).values())

    def attention(**kw):
        r = svd.tree_attention(q, c, tab, ctx, want_lse=True, **kw)
        return r["out"], r["lse"]

    def read(**kw):
        return svd.cache_read(c, tab, 300, start=start, **kw)

    def adjust(**kw):
        return (svd.adjust_logits(z, h, hlen, frequency=f, **kw),)

    return [("tree", tree), ("attention", attention), ("read", read), ("adjust", adjust)]


def verification_calls(svd):
    torch.manual_seed(6)
    B, K, G, V = 3, 2, 4, 20011
    p = torch.randn(B, K, G + 1, V, device="cuda")
    q = torch.randn(B, K, G, V, device="cuda")
    d = torch.randint(0, V, (B, K, G), dtype=torch.int32, device="cuda")
    p1, q1, d1 = (x[:, 0].contiguous() for x in (p, q, d))
    px = torch.arange(B * K * (G + 1), dtype=torch.int32, device="cuda").view(B, K, G + 1)
    qx = torch.arange(B * K * G, dtype=torch.int32, device="cuda").view(B, K, G)
    pp, qp = p.view(-1, V), q.view(-1, V)
    lat = svd.cps_lattice(q1)
    first, length, avg = i32(0, 1, 0), i32(2, 4, 1), torch.zeros((B, 2), dtype=torch.int32, device="cuda")

    def call(f, *a, **fixed):
        def run(**kw):
            r = f(*a, **fixed, **kw)
            return tuple(x for x in (r.values() if isinstance(r, dict) else (r,)) if x is not None)
        return run

    return [("select", call(svd.select_and_verify, p, q, d, want_alpha=True, want_beta=True)),
            ("verify", call(svd.verify, p1, q1, d1, want_alpha=True)),
            ("greedy_select", call(svd.greedy_select_and_verify, p, d, want_alpha=True)),
            ("greedy", call(svd.greedy_verify, p1, d1)),
            ("rows", call(svd.select_and_verify_rows, pp, px, qp, qx, d)),
            ("window", call(svd.verify_window, p, q, d, gamma_b=length)),
            ("lattice", call(svd.cps_lattice, q1)),
            ("beam", call(svd.cps_beam, lat)),
            # shift = 0: the window follows the last step alone, so that every call gives the same
            ("adl", call(svd.adl_next, d, first, length, avg, shift=0))]


def calls(svd):
    return step_calls(svd) + verification_calls(svd)


def storages(r):
    return {x.untyped_storage().data_ptr(): x.untyped_storage().nbytes() for x in r}


NAMES = ["tree", "attention", "read", "adjust", "select", "verify", "greedy_select", "greedy", "rows",
         "window", "lattice", "beam", "adl"]


@pytest.fixture(params=NAMES)
def job(request):
    svd = require_gpu()
    say(request.param)
    return svd, dict(calls(svd))[request.param]


def test_results_on_another_stream(job):
    svd, call = job
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, torch.cuda.current_stream().cuda_stream, 0):
        torch.cuda.synchronize()
        got = call(stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_results_are_not_put_into_memory_in_use(job):
    # blocks as large as the results, dropped while a copy of each still waits
    svd, call = job
    sizes = storages(call())
    torch.cuda.synchronize()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes.values()]
    copies = [torch.empty_like(x) for x in held]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(SPIN)
    for x, y in zip(held, copies):
        y.copy_(x)
    del held, x, y
    got = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    for y in copies:
        assert (y == 7).all()
    want = call()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_dropped_results_go_back_after_the_call(job):
    # results dropped at once: new memory of the current stream is not theirs while the call waits
    svd, call = job
    sizes = storages(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    call(stream=side.cuda_stream)
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes.values()]
    torch.cuda.synchronize()
    for x in held:
        assert (x == 7).all()


def test_what_a_call_allocates_lasts_as_long_as_the_call(job, monkeypatch):
    svd, call = job
    want = [x.clone() for x in call()]
    made, empty = [], torch.empty

    def spy(*a, **kw):
        t = empty(*a, **kw)
        made.append((t.data_ptr(), max(t.numel() * t.element_size(), 1)))
        return t

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    monkeypatch.setattr(torch, "empty", spy)
    got = call(stream=side.cuda_stream)
    monkeypatch.undo()
    fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(4)]
    taken = {x.data_ptr() for x in fill}
    assert not any(at in taken for at, _ in made)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for x in fill:
        assert (x == 0xFF).all()


def test_a_cache_write_on_another_stream():
    svd = require_gpu()
    c = svd.kv_cache(4, 2, 16, 64)
    tab = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    ctx = i32(5)
    k = torch.randn(1, 50, 2, 64, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    svd.cache_write(c, k, -k, tab, ctx, stream=side.cuda_stream)
    torch.cuda.synchronize()
    gk, gv = svd.cache_read(c, tab, 50, start=i32(5))
    assert torch.equal(gk, k) and torch.equal(gv, -k)
