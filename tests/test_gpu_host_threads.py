"""Calls from host threads that have not called CUDA before, with every array given: what the main thread gets."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def in_a_new_thread(fn):
    """(status, message) of an entry's call."""
    import linear_attention_sequence_rule_b200 as gdn
    got = []
    t = threading.Thread(target=lambda: got.append((fn(), gdn.gdn_last_error())))
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts(d, dtype):
    import linear_attention_sequence_rule_b200 as gdn
    T, code = 300, gdn._DT[DT[dtype]]
    g = torch.Generator("cuda").manual_seed(d)
    q, do = (torch.randn(1, T, 4, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    k, v = (torch.randn(1, T, 2, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    out, lse = gdn.attn_fwd(q, k, v, scale=0.125)
    want = [out, lse, *gdn.attn_bwd(q, k, v, out, lse, do, scale=0.125)]
    got = [torch.zeros_like(x) for x in want]
    ws = torch.empty(gdn.gdn_attn_bwd_workspace_bytes(1, T, 4, 2, d, 0, code), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    p = [x.data_ptr() for x in got]
    ins = [x.data_ptr() for x in (q, k, v)]
    ddo, dws, n = do.data_ptr(), ws.data_ptr(), ws.numel()
    rc = in_a_new_thread(lambda: gdn.gdn_attn_fwd(*ins, p[0], p[1], 1, T, 4, 2, d, None, code, 0.125, 0))
    assert rc == (gdn.GDN_OK, "")
    rc = in_a_new_thread(lambda: gdn.gdn_attn_bwd(*ins, p[0], p[1], ddo, *p[2:], 1, T, 4, 2, d, None, code, 0.125, dws, n, 0))
    assert rc == (gdn.GDN_OK, "")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_generation_step(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    N, Hq, Hk, d, page, blocks, P, code = 3, 4, 2, 64, 32, 4, 20, gdn._DT[DT[dtype]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    lens, added, free, head = i32([0] * N), i32([70, 1, 40]), i32(list(range(P))), i32([0])
    rows = 111
    k, v = (torch.randn(rows, Hk, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = torch.randn(N, Hq, d, generator=g, device="cuda").to(DT[dtype])

    def arrays():
        return dict(table=i32([[-1] * blocks] * N), cu=i32([0] * (N + 1)), slots=i32([0] * rows), pos=i32([0] * rows),
                    lens=i32([0] * N), head=i32([0]), status=i32([9, 9]),
                    kc=torch.zeros(P, Hk, page, d, dtype=torch.uint8, device="cuda"),
                    vc=torch.zeros(P, Hk, page, d, dtype=torch.uint8, device="cuda"),
                    ks=torch.zeros(P, Hk, device="cuda"), vs=torch.zeros(P, Hk, device="cuda"), out=torch.zeros_like(q))

    def calls(a):
        p = {x: y.data_ptr() for x, y in a.items()}
        i = [x.data_ptr() for x in (lens, added, free, head, k, v, q)]
        return [lambda: gdn.gdn_cache_plan(i[0], i[1], p["table"], i[2], i[3], p["cu"], p["slots"], p["pos"], p["lens"],
                                           p["head"], p["status"], N, blocks, P, rows, page, 0),
                lambda: gdn.gdn_cache_append(i[4], i[5], p["slots"], p["kc"], p["vc"], p["ks"], p["vs"], rows, Hk, d, page, P,
                                             code, 0),
                lambda: gdn.gdn_attn_decode(i[6], p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], p["out"], N, Hq,
                                            Hk, d, page, P, blocks, code, 0.125, None, 0, 0)]

    assert gdn.gdn_attn_decode_workspace_bytes(N, Hq, Hk, d, page, blocks, code) == 0
    want, got = arrays(), arrays()
    torch.cuda.synchronize()
    for fn in calls(want):
        assert fn() == gdn.GDN_OK, gdn.gdn_last_error()
    torch.cuda.synchronize()
    for fn in calls(got):
        assert in_a_new_thread(fn) == (gdn.GDN_OK, "")
    assert want["status"].tolist() == [0, 0] and all(torch.equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_forward(dtype):
    import linear_attention_sequence_rule_b200 as gdn
    T, H, d, code = 200, 2, 64, gdn._DT[DT[dtype]]
    g = torch.Generator("cuda").manual_seed(2)
    q, k, v = (torch.nn.functional.normalize(torch.randn(1, T, H, d, generator=g, device="cuda"), dim=-1).to(DT[dtype])
               for _ in range(3))
    la, be = -0.1 * torch.rand(1, T, H, generator=g, device="cuda"), torch.rand(1, T, H, generator=g, device="cuda")
    want = gdn.chunk_fwd(q, k, v, la, be)
    got = [torch.zeros_like(x) for x in want]
    ws = torch.empty(max(256, gdn.gdn_chunk_fwd_workspace_bytes(1, T, H, d, d, 64, 0, code)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    ins, outs = [x.data_ptr() for x in (q, k, v, la, be)], [x.data_ptr() for x in got]
    pw, n = ws.data_ptr(), ws.numel()
    rc = in_a_new_thread(lambda: gdn.gdn_chunk_fwd(*ins, None, *outs, 1, T, H, d, d, 64, None, code, pw, n, 0))
    assert rc == (gdn.GDN_OK, "")
    assert all(torch.equal(a, b) for a, b in zip(got, want))
