"""The time-out path of the tensor-core kernels, made to run on purpose.

Every mbarrier wait in the tcgen05 kernels is bounded; when one runs out the
kernel records DA_DEVERR_TIMEOUT, every role leaves its loop, the copies in
flight and the tensor-core work are drained and tensor memory is freed, so
the context stays usable.  The DA_FLAG_TEST_STALL hook makes the MMA-issuing
thread of every CTA wait first on a barrier that nothing signals (2 ms
limit), which drives each role into that path from a known point: copies
issued, nothing consumed.  The tests check the error word, and that a normal
call on the same buffers right after it returns the clean result bit for bit
(a CTA that left tensor memory allocated, or an arrival still in flight into
freed shared memory, would show up there or hang the next launch's
allocation).  The CPU test checks the flag's validation.
"""

import pytest
import torch

from invariant_decode_attention_gb300 import workloads as W

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


def _workloads():
    return {
        "mla": W.make(W.INDEXED, [40, 300, 1500, 2048], H_q=128, H_kv=1, D_qk=576, D_v=512,
                      latent=True, num_slots=4096, seed=71),
        "mla_fp8": W.quantize_fp8(W.make(W.INDEXED, [40, 300, 1500, 2048], H_q=128, H_kv=1,
                                         D_qk=576, D_v=512, latent=True, num_slots=4096,
                                         seed=76)),
        "gqa_tc": W.make(W.PAGED, [40, 300, 1500, 5000], H_q=64, H_kv=2, D_qk=128,
                         page_size=16, seed=72),
        "gqa_tc_fp8": W.quantize_fp8(W.make(W.PAGED, [40, 300, 1500, 5000], H_q=64, H_kv=2,
                                            D_qk=128, page_size=16, seed=73)),
        "gqa_tc_nvfp4": W.nvfp4_kv(W.make(W.PAGED, [40, 300, 1500, 5000], H_q=64, H_kv=2,
                                          D_qk=128, page_size=16, seed=74, draw_kv=False),
                                   seed=75),
    }


def test_flag_validation(api):
    wl = _workloads()["gqa_tc"]
    prob = api.problem_for(wl)
    prob.flags = api.FLAG_TEST_STALL
    assert api.workspace_bytes(prob) > 0
    prob.flags = 2
    with pytest.raises(RuntimeError):
        api.workspace_bytes(prob)


@gpu
@pytest.mark.parametrize("kind", ["mla", "mla_fp8", "gqa_tc", "gqa_tc_fp8", "gqa_tc_nvfp4"])
def test_stall_times_out_and_context_stays_usable(api, kind):
    wl = _workloads()[kind]
    g = wl.to("cuda")
    prob = api.problem_for(g)
    variant = api.split_constants(prob)[0]
    assert variant == (api.VARIANT_MLA if kind.startswith("mla") else api.VARIANT_GQA_TC)
    o_ref, l_ref = [t.clone() for t in api.run_workload(g)]

    prob.flags = api.FLAG_TEST_STALL
    ws = api.workspace(prob)
    out = torch.empty((g.B, g.H_q, g.D_v), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((g.B, g.H_q), dtype=torch.float32, device="cuda")
    for _ in range(2):  # twice: the first stalled call left nothing behind
        pl = api.plan(prob, api.INVARIANT, g.lengths, ws)
        api.run(pl, g.q, g.k, g.v, g.table, g.lengths, out, lse)
        api.combine(pl, out, lse)
        err = api.read_error(pl)
        assert err & api.DEVERR_TIMEOUT, err
        assert not err & (api.DEVERR_INDEX | api.DEVERR_LENGTH), err

    for _ in range(2):
        o, l = api.run_workload(g, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(o, o_ref) and torch.equal(l, l_ref)


@gpu
@pytest.mark.parametrize("n,max_rank,x_dtype", [(90, 64, 1), (90, 128, 0), (1300, 64, 0), (1300, 128, 1)])
def test_stalled_adapters_time_out_and_the_next_call_is_clean(api, n, max_rank, x_dtype):
    """nvfp4_mm_adapters with the first stage of one of its two matmul kernels never full:
    one issuing thread waits for it (2 ms limit) while the other one goes on, with
    commits to every kind of barrier behind it."""
    g = torch.Generator().manual_seed(n + max_rank)
    N, K, count = 1024, 2176, 3
    x = torch.randn((n, K), generator=g).to(torch.bfloat16 if x_dtype else torch.float32).cuda()
    y = torch.randn((n, N), generator=g).cuda()
    a = (torch.randn((count, max_rank, K), generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    b = torch.randn((count, N, max_rank), generator=g).to(torch.bfloat16).cuda()
    ids = torch.sort(torch.randint(-1, count, (n,), generator=g, dtype=torch.int32))[0].cuda()
    h = api.Adapters(a, b)
    ws = api.adapters_workspace(n, N, K, h)
    want = api.nvfp4_adapters(x, h, ids, y, out=torch.empty_like(y), ws=ws)
    assert api.nvfp4_read_error(ws) == 0
    out = torch.empty_like(y)

    def call(flag):
        status = api.lib().nvfp4_mm_adapters(
            x.data_ptr(), x_dtype + flag, n, N, K, a.data_ptr(), b.data_ptr(), count, max_rank, None,
            None, ids.data_ptr(), y.data_ptr(), out.data_ptr(), None, ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert status == api.OK
        return api.nvfp4_read_error(ws)
    for flag in (api.X_TEST_STALL_DOWN, api.X_TEST_STALL_UP):
        for _ in range(2):  # twice: the first stalled call left nothing behind
            assert call(flag) == api.DEVERR_TIMEOUT
        for _ in range(2):
            out.fill_(float("nan"))
            assert call(0) == 0
            assert torch.equal(out, want)


def test_adapters_flag_validation(api):
    fake = 1 << 20  # never dereferenced: every case fails before any device work

    def call(x_dtype):
        return api.lib().nvfp4_mm_adapters(fake, x_dtype, 4, 128, 64, fake, fake, 2, 16, None, None,
                                           fake, 1 << 24, 1 << 28, None, fake, 0, None)
    for good in (0, 1, 0x100, 0x101, 0x200, 0x201):
        assert call(good) == api.ERR_WORKSPACE, good
    for bad in (2, 0x102, 0x202, 0x300, 0x301, -1, -256, -255):
        assert call(bad) == api.ERR_INVALID_ARG, bad
