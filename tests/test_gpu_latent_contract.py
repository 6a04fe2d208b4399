"""What the latent operators promise around their results: the same bits from every run, waits that run out
and leave the cache alone, statuses of replayed graphs, streams, scratch and arguments of other types."""
import numpy as np
import pytest
import torch

from oracle import latent_attention as la
from test_gpu_latent import (B, SCALE, Cache, _check_decode, _check_prefill, _ints, _prefill_inputs,  # noqa: F401
                             _queries)
from test_latent_contract import check_lse, check_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,qs,ks", [(16, [300, 1, 90, 700], [300, 129, 90, 1400]), (4, [2048], [4096])])
def test_prefill_repeats_bit_for_bit(B, H, qs, ks):  # noqa: F811
    """Copies, products and the softmax meet at barriers of both CTAs of a pair: no result may depend on who came
    first."""
    q, kv, kp, dev, cu = _prefill_inputs(qs, ks, H, seed=81, joint=True)
    first, lse1 = B.latent_attention_prefill(*dev, SCALE)
    runs = [B.latent_attention_prefill(*dev, SCALE) for _ in range(40)]
    assert B.latent_last_status() == 0
    for out, lse in runs:
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), lse1.view(torch.int32))
    if sum(ks) < 2000:
        _check_prefill(q, kv, kp, cu, first, lse1, True)


@pytest.mark.parametrize("indexer,joint", [(False, False), (True, True)])
def test_eviction_whose_wait_ran_out_leaves_the_slots_alone(B, indexer, joint):  # noqa: F811
    """With a test option the first 64 kept keys of a sequence never count as read, so that what waits for them
    (limit 50 ms here) runs out: it is reported, and those slots keep their keys."""
    lens, budget, recent = [400, 250, 330], 256, 20
    c = Cache(lens, seed=82, joint=joint)
    g = torch.Generator().manual_seed(83)
    w = torch.rand((3, c.table.shape[1] * 64), generator=g)
    w[:, :64] = 0.0  # the first 64 keys go, so that chunk 0 keeps keys that live in chunk 1's slots
    kc = torch.randint(0, 256, (c.P, 64, 128), generator=g, dtype=torch.uint8)
    ks = torch.rand((c.P, 64), generator=g)
    ck, kp = c.device()
    dw, dk, ds = w.cuda(), kc.cuda() if indexer else None, ks.cuda() if indexer else None
    B.set_option("wait_limit_us", 50000)
    B.set_option("test_withhold", 1)
    try:
        kept, new = B.latent_cache_evict(ck, kp, dw, c.table.cuda(), _ints(lens), budget, recent, k_cache=dk,
                                         k_cache_scale=ds)
        assert B.latent_last_status() == B.DSA_ERR_TIMEOUT
    finally:
        B.set_option("test_withhold", 0)
        B.set_option("wait_limit_us", 2000000)
    assert new.tolist() == [256, 250, 256]
    want = c.data.clone().view(torch.int16).reshape(-1, 576)
    old, wk, ws = want.clone(), kc.clone().reshape(-1, 128), ks.clone().reshape(-1)
    for b, L in enumerate(lens):
        rows = la.kept_keys(w[b].numpy(), L, budget, recent)
        assert np.array_equal(kept[b, :len(rows)].cpu().numpy(), rows)
        if L <= budget:
            continue
        assert rows[0] >= 64  # (or nothing here would have to wait)
        # the chunks that hold some of the first 64 kept keys in their own slots
        waits = {int(r) // 64 for r in rows[:64]} - {0}
        assert waits and max(waits) < budget // 64
        slots = torch.from_numpy(la.slots_of(c.table[b].numpy(), L))
        for i, r in enumerate(rows):
            if i // 64 in waits:
                continue
            want[slots[i]] = old[slots[r]]
            wk[slots[i]] = kc.reshape(-1, 128)[slots[r]]
            ws[slots[i]] = ks.reshape(-1)[slots[r]]
    assert torch.equal(ck.cpu().contiguous().view(torch.int16).reshape(-1, 512), want[:, :512])
    assert torch.equal(kp.cpu().contiguous().view(torch.int16).reshape(-1, 64), want[:, 512:])
    if indexer:
        assert torch.equal(dk.cpu().reshape(-1, 128), wk) and torch.equal(ds.cpu().reshape(-1), ws)
    # the next call is a whole one again
    kept, new = B.latent_cache_evict(ck, kp, dw, c.table.cuda(), _ints([256, 250, 256]), 100, 7)
    assert B.latent_last_status() == 0 and new.tolist() == [100, 100, 100]


def test_an_evictions_time_out_is_never_lost(B):  # noqa: F811
    """Waits that run out at once report beside the chunk that collects the call's status, in any order; a bad page is
    reported as well, and the next call starts from no status."""
    lens, budget = [400] * 24, 256
    c = Cache(lens, seed=84)
    table, dl = c.table.cuda(), _ints(lens)
    w = torch.ones((24, c.table.shape[1] * 64))
    w[:, :64] = 0.0
    ck, kp = c.device()
    B.set_option("wait_limit_us", 1)
    B.set_option("test_withhold", 1)
    try:
        for _ in range(200):
            B.latent_cache_evict(ck, kp, w.cuda(), table, dl, budget, 20)
            assert B.latent_last_status() == B.DSA_ERR_TIMEOUT
    finally:
        B.set_option("test_withhold", 0)
        B.set_option("wait_limit_us", 2000000)
    bad = c.table.clone()
    bad[3, 1] = c.P
    B.latent_cache_evict(ck, kp, w.cuda(), bad.cuda(), dl, budget, 20)
    assert B.latent_last_status() == B.DSA_ERR_RANGE
    B.latent_cache_evict(ck, kp, w.cuda(), table, dl, budget, 20)
    assert B.latent_last_status() == 0


def _capture(stream, call):
    """call() once on the stream, which sizes its scratch, then into a graph."""
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
    return g


def test_a_graphs_status_outlives_the_scratch_it_was_captured_with(B):  # noqa: F811
    c, big = Cache([300, 64], seed=85), Cache([4000] * 8, seed=86)
    qn, qp = (x.cuda() for x in _queries(2, 1, 16, seed=87))
    qbn, qbp = (x.cuda() for x in _queries(8, 2, 64, seed=88))
    (ck, kp), table, lens = c.device(), c.table.cuda(), _ints(c.lens)
    (bck, bkp), btable, blens = big.device(), big.table.cuda(), _ints(big.lens)
    w = torch.zeros((8, big.table.shape[1] * 64), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(qn), torch.empty((2, 1, 16), device="cuda")
    g = _capture(s, lambda: B.latent_attention_paged(qn, qp, ck, kp, table, lens, SCALE, out=out, lse=lse))
    with torch.cuda.stream(s):  # a larger call replaces the scratch
        B.latent_attention_paged(qbn, qbp, bck, bkp, btable, blens, SCALE, weights=w)
    assert B.latent_last_status(s) == 0
    lens.copy_(_ints([300, 10 ** 6]))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.replay()
    assert B.latent_last_status(s) == B.DSA_ERR_RANGE
    lens.copy_(_ints(c.lens))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.replay()
    assert B.latent_last_status(s) == 0
    _check_decode(c, qn.cpu(), qp.cpu(), out.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("scale", [np.float32(SCALE), np.float64(SCALE), torch.tensor(SCALE), 1])
def test_scales_of_other_number_types(B, scale):  # noqa: F811
    c = Cache([70, 3], seed=89)
    qn, qp = (x.cuda() for x in _queries(2, 1, 16, seed=90))
    (ck, kp), table, lens = c.device(), c.table.cuda(), _ints(c.lens)
    _, _, _, dev, _ = _prefill_inputs([20], [30], 2, seed=91, joint=True)
    calls = [lambda s: B.latent_attention_paged(qn, qp, ck, kp, table, lens, s),
             lambda s: B.latent_attention_shared_prefix(qn, qp, ck, kp, table[0, :1].contiguous(), _ints([5]), table,
                                                        lens, s),
             lambda s: B.latent_attention_prefill(*dev, s)]
    for call in calls:
        for x, y in zip(call(scale), call(float(scale))):
            assert torch.equal(x, y)


@pytest.mark.parametrize("mode", ["global", "relaxed"])
def test_a_call_that_has_to_grow_the_scratch_leaves_a_capture_whole(B, mode):  # noqa: F811
    c = Cache([70, 3], seed=92)
    qn, qp = (x.cuda() for x in _queries(2, 1, 16, seed=93))
    (ck, kp), table, lens = c.device(), c.table.cuda(), _ints(c.lens)
    out, lse, x = torch.empty_like(qn), torch.empty((2, 1, 16), device="cuda"), torch.zeros(5, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call():
        B.latent_attention_paged(qn, qp, ck, kp, table, lens, SCALE, out=out, lse=lse)

    B.release()  # no stream has scratch now
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s, capture_error_mode=mode):
        with pytest.raises(B.IndexerError) as e:
            call()
        x.add_(1.0)
    assert e.value.code == B.DSA_ERR_CUDA
    g.replay()
    torch.cuda.synchronize()
    assert torch.all(x == 1.0) and B.latent_last_status(s) == 0
    g = _capture(s, call)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    _check_decode(c, qn.cpu(), qp.cpu(), out.double().cpu().numpy(), lse.double().cpu().numpy())


def _freed_while_in_use(shape, dtype, fill):
    """Gives a tensor's memory back while the current stream has yet to write it."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda._sleep(40_000_000)  # some 20 ms
    x.fill_(fill)


def test_outputs_of_a_call_on_a_given_stream_lie_in_its_memory(B):  # noqa: F811
    """An output taken from the current stream's memory would be written by another stream while that memory's last
    user, here a slow fill, still runs."""
    lens = [70] * 40
    c = Cache(lens, seed=94)
    qn, qp = (x.cuda() for x in _queries(40, 1, 16, seed=95))
    (ck, kp), table, dl = c.device(), c.table.cuda(), _ints(lens)
    q, kv, kpe, dev, cu = _prefill_inputs([90], [90], 16, seed=96, joint=True)
    w = torch.rand((40, c.table.shape[1] * 64), generator=torch.Generator().manual_seed(97))
    dw, s = w.cuda(), torch.cuda.Stream()
    B.latent_attention_paged(qn, qp, ck, kp, table, dl, SCALE, stream=s)  # (scratch, and this stream's memory)
    B.latent_attention_prefill(*dev, SCALE, stream=s)
    torch.cuda.synchronize()
    _freed_while_in_use(tuple(qn.shape), torch.bfloat16, 7.0)
    out, lse = B.latent_attention_paged(qn, qp, ck, kp, table, dl, SCALE, stream=s)
    torch.cuda.synchronize()
    _check_decode(c, qn.cpu(), qp.cpu(), out.double().cpu().numpy(), lse.double().cpu().numpy())
    _freed_while_in_use((90, 16, 128), torch.bfloat16, 7.0)
    out, lse = B.latent_attention_prefill(*dev, SCALE, stream=s)
    torch.cuda.synchronize()
    _check_prefill(q, kv, kpe, cu, out, lse, True)
    _freed_while_in_use((40, 65), torch.int32, 7)
    kept, new = B.latent_cache_evict(ck, kp, dw, table, dl, 65, 3, stream=s)
    torch.cuda.synchronize()
    for b in range(40):
        assert np.array_equal(kept[b].cpu().numpy(), la.kept_keys(w[b].numpy(), 70, 65, 3))


def _odd(t):
    """The same elements with strides of 1, 3 or 5 on the axes of one element."""
    return t.as_strided(t.shape, [s if n > 1 else 1 + 2 * i for i, (n, s) in enumerate(zip(t.shape, t.stride()))])


@pytest.mark.parametrize("H,qs,ks", [(1, [1], [1]), (1, [40], [70]), (3, [1], [70]), (2, [1], [1])])
def test_prefill_takes_any_stride_of_an_axis_of_one(B, H, qs, ks):  # noqa: F811
    q, kv, kpe, dev, cu = _prefill_inputs(qs, ks, H, seed=98, joint=True)
    odd = [_odd(t) for t in dev[:4]]
    odd[2] = dev[2].as_strided((ks[0], 64), (64 if ks[0] > 1 else 3, 1))
    out, lse = B.latent_attention_prefill(*odd, *dev[4:], SCALE)
    _check_prefill(q, kv, kpe, cu, out, lse, True)
    with pytest.raises(B.IndexerError):  # where an axis is stepped along, its stride has to be a multiple of 8
        wide = torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
        B.latent_attention_prefill(wide.as_strided((2, H, 192), (4, 192, 1)), *dev[1:], SCALE)


def test_scratch_of_many_sequences_is_that_of_the_cut_ones(B):  # noqa: F811
    """600 sequences of 128 heads: 1200 row blocks, of which the 152 CTAs' runs cut two per CTA at most, 128 KB each.
    (Slots for all of them would be 177 MB.)"""
    lens = [1 + (37 * i) % 150 for i in range(600)]
    c = Cache(lens, seed=99)
    qn, qp = _queries(600, 1, 128, seed=100)
    dq, dp = qn.cuda(), qp.cuda()
    (ck, kp), table, dl = c.device(), c.table.cuda(), _ints(lens)
    out, lse = torch.empty_like(dq), torch.empty((600, 1, 128), device="cuda")
    B.latent_attention_paged(dq[:1], dp[:1], ck, kp, table[:1], dl[:1], SCALE)  # the kernels are loaded
    torch.cuda.synchronize()
    B.release()
    before = torch.cuda.mem_get_info()[0]
    B.latent_attention_paged(dq, dp, ck, kp, table, dl, SCALE, out=out, lse=lse)
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] <= 64 << 20
    assert B.latent_last_status() == 0
    _check_decode(c, qn, qp, out.double().cpu().numpy(), lse.double().cpu().numpy(), only=range(0, 600, 7))


def test_graphs_captured_on_streams_of_their_own_run_side_by_side(B):  # noqa: F811
    """Both cut into pieces that meet in scratch; each has its own, so replays may overlap."""
    ins = []
    for i, (lens, H) in enumerate((([3000, 2500], 16), ([2000, 70, 900], 64))):
        c = Cache(lens, seed=101 + i)
        qn, qp = (x.cuda() for x in _queries(len(lens), 1, H, seed=103 + i))
        (ck, kp), table, dl = c.device(), c.table.cuda(), _ints(lens)
        out, lse = torch.empty_like(qn), torch.empty((len(lens), 1, H), device="cuda")
        w = torch.zeros((len(lens), c.table.shape[1] * 64), device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())

        def call(a=(qn, qp, ck, kp, table, dl, SCALE), o=out, z=lse, w=w):
            w.zero_()
            B.latent_attention_paged(*a, out=o, lse=z, weights=w)

        # (the call's arguments live as long as its graph)
        ins.append((_capture(s, call), (out, lse, w), torch.cuda.Stream(), call, (c, qn.cpu(), qp.cpu()), s))
    alone = []
    for g, res, _, _, (c, qn, qp), s in ins:
        g.replay()
        torch.cuda.synchronize()
        assert B.latent_last_status(s) == 0
        out, lse, w = (t.double().cpu().numpy() for t in res)
        _check_decode(c, qn, qp, out, lse, weights=w)
        alone.append([t.clone() for t in res])
    for _ in range(30):
        for _, res, *_ in ins:
            for t in res:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for g, _, s, *_ in ins:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (_, res, *_), want in zip(ins, alone):
            assert all(torch.equal(x, y) for x, y in zip(res, want))


@pytest.mark.parametrize("nn,H,lens", [(1, 16, [200]), (1, 128, [2100, 64]), (1, 16, [30000]), (2, 24, [640, 700]),
                                       (4, 5, [4000, 130])])
def test_key_weights_and_lse_have_the_bits_of_fp32(B, nn, H, lens):  # noqa: F811
    c = Cache(lens, seed=110 + H)
    qn, qp = _queries(len(lens), nn, H, seed=111 + nn)
    (ck, kp), table, dl = c.device(), c.table.cuda(), _ints(lens)
    w = torch.zeros((len(lens), c.table.shape[1] * 64), device="cuda")
    _, lse = B.latent_attention_paged(qn.cuda(), qp.cuda(), ck, kp, table, dl, SCALE, weights=w)
    _, lse1 = B.latent_attention_paged(qn.cuda(), qp.cuda(), ck, kp, table, dl, SCALE)
    ckv, kpe = c.flat()
    ref = la.decode(qn.double().numpy(), qp.double().numpy(), ckv, kpe, c.table.numpy(), lens, SCALE)
    for b, L in enumerate(lens):
        check_weights(w[b, :L].double().cpu().numpy(), ref[b][2])
        for x in (lse, lse1):
            check_lse(x[b].double().cpu().numpy().reshape(-1), ref[b][1])


@pytest.mark.parametrize("H,qs,ks", [(4, [300, 70], [300, 700]), (2, [1000], [1500])])
def test_prefill_lse_has_the_bits_of_fp32(B, H, qs, ks):  # noqa: F811
    q, kv, kpe, dev, cu = _prefill_inputs(qs, ks, H, seed=112, joint=True)
    _, lse = B.latent_attention_prefill(*dev, SCALE)
    lse = lse.double().cpu().numpy()
    for z in range(len(qs)):
        (a, b), (m, n) = cu[0][z:z + 2], cu[1][z:z + 2]
        sees = (n - m) - (b - a) + 1 + np.arange(b - a)
        for h in range(H):
            k = np.concatenate([kv[m:n, h, :128].double().numpy(), kpe[m:n].double().numpy()], 1)
            ref = la.rows_over_keys(q[a:b, h].double().numpy(), k, k[:, :1], sees, SCALE)
            check_lse(lse[a:b, h], ref[1])


def test_any_object_that_names_a_stream(B):  # noqa: F811
    class Raw:
        def __init__(self, handle):
            self.cuda_stream = handle

    c = Cache([70, 3], seed=113)
    qn, qp = (x.cuda() for x in _queries(2, 1, 16, seed=114))
    (ck, kp), table, dl = c.device(), c.table.cuda(), _ints(c.lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (Raw(s.cuda_stream), Raw(0), s):
        out, lse = B.latent_attention_paged(qn, qp, ck, kp, table, dl, SCALE, stream=stream)
        torch.cuda.synchronize()
        _check_decode(c, qn.cpu(), qp.cpu(), out.double().cpu().numpy(), lse.double().cpu().numpy())
