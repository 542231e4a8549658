"""Layer norm, gated recurrence and gradient clipping where offsets pass 32
bits, and in two streams at once.  What is compared is the same call on small
contiguous tensors, bit for bit (its values are tested elsewhere)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


@pytest.fixture
def room():
    """A function that gives device memory for a test, or skips it."""
    def give(numel, dtype):
        free, _ = torch.cuda.mem_get_info()
        if numel * torch.empty(0, dtype=dtype).element_size() > free // 2:
            pytest.skip("not enough device memory")
        return torch.empty(numel, dtype=dtype, device="cuda")
    yield give
    torch.cuda.empty_cache()


def _rows(wide, T, pitch, at, C):
    return wide[: T * pitch].view(T, pitch)[:, at:at + C]


@pytest.mark.parametrize("odd", [0, 1])
def test_rows_beyond_32_bits(A, room, odd):
    T, C, dt = 70, 200, torch.bfloat16
    pitch = (1 << 25) + odd            # row 64 begins at element 2^31
    wide = room(T * pitch, dt)
    g = torch.Generator(device="cuda").manual_seed(odd)
    ins = [torch.randn(T, C, generator=g, device="cuda").to(dt) for _ in range(4)]
    far = [_rows(wide, T, pitch, 1000 * i, C) for i in range(8)]
    for t, v in zip(far, ins):
        t.copy_(v)
    near_out = [torch.empty(T, C, dtype=dt, device="cuda") for _ in range(4)]
    gain = torch.randn(C, generator=g, device="cuda")
    results = []
    for (x, f, gate, dy), (out, dx, df, dg) in ((ins, near_out), (far[:4], far[4:])):
        fin, d0 = torch.empty(2, 1, C, device="cuda")
        chunk = torch.empty(2, C, device="cuda")
        A.attnres_gated_recurrence(x, f, out, gate=gate, final_state=fin, chunk_states=chunk)
        A.attnres_gated_recurrence_backward(x, f, chunk, dy, dx, df, dg, gate=gate, grad_initial_state=d0)
        got = [t.clone() for t in (out, dx, df, dg, fin, d0)]
        gg, gb = torch.empty(2, C, device="cuda")
        A.attnres_layer_norm(x, out, gain)
        A.attnres_layer_norm_backward(x, dy, dx, gain, gg, gb)
        results.append(got + [out.clone(), dx.clone(), gg, gb])
    for i, (near, away) in enumerate(zip(*results)):
        if i < 6 or not odd:
            assert torch.equal(near, away)
        else:  # off the vectors a layer norm adds its row in another order: C fp32 roundings, and that of the result
            assert torch.allclose(near.float(), away.float(), rtol=2 ** -7, atol=C * 2 ** -20)


def test_slots_beyond_32_bits(A, room):
    C, slots = 1 << 16, 33000
    state = room(slots * C, torch.float32).view(slots, C)
    x, f, gate = torch.randn(3, 2, C, device="cuda")
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    start = torch.randn(2, C, device="cuda")
    state[at.long()] = start
    out, want = torch.empty(2, 2, C, device="cuda")
    A.attnres_gated_recurrence_step(x, f, state, out, gate=gate, slots=at)
    A.attnres_gated_recurrence_step(x, f, start, want, gate=gate)
    assert torch.equal(out, want) and torch.equal(state[at.long()], start)


def test_a_gradient_beyond_32_bits(A, room):
    n = (1 << 31) + 77
    grad = room(n, torch.bfloat16)
    grad.zero_()
    grad[5], grad[1 << 31], grad[n - 1] = 2.0, -4.0, 4.0   # norm 6
    norm = torch.empty(1, device="cuda")
    A.attnres_grad_clip([grad], 1.5, norm)
    assert norm.item() == 6.0
    assert grad[[5, 1 << 31, n - 1]].tolist() == [0.5, -1.0, 1.0]
    assert torch.count_nonzero(grad[-100:]).item() == 2 and torch.count_nonzero(grad[:100]).item() == 1


def test_two_streams_at_once(A):
    """Calls of every operator in flight on two streams: no state is shared."""
    dt, T, C, n = torch.bfloat16, 6000, 1032, 4
    cu = torch.tensor([0, 1000, 1003, 4500, T], dtype=torch.int32, device="cuda")

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = [torch.randn(T, C, generator=g, device="cuda").to(dt) for _ in range(4)]
        r = dict(x=t[0], f=t[1], g=t[2], dy=t[3], s0=torch.randn(n, C, generator=g, device="cuda"))
        r["gain"] = torch.randn(C, generator=g, device="cuda")
        for k in ("out", "dx", "df", "dg", "h", "dh"):
            r[k] = torch.zeros(T, C, dtype=dt, device="cuda")
        r["fin"], r["d0"] = torch.zeros(2, n, C, device="cuda")
        r["chunk"] = torch.zeros(-(-T // 64), C, device="cuda")
        r["gg"], r["gb"] = torch.zeros(2, C, device="cuda")
        r["norm"] = torch.zeros(1, device="cuda")
        r["ws"] = torch.empty(A.attnres_layer_norm_backward_workspace_size(T, C), dtype=torch.uint8, device="cuda")
        r["cws"] = torch.empty(A.attnres_grad_clip_workspace_size(), dtype=torch.uint8, device="cuda")
        return r

    def call(r, s):
        A.attnres_layer_norm(r["x"], r["h"], r["gain"], stream=s)
        A.attnres_gated_recurrence(r["h"], r["f"], r["out"], gate=r["g"], cu_seqlens=cu, initial_state=r["s0"], final_state=r["fin"],
                                   chunk_states=r["chunk"], stream=s)
        A.attnres_gated_recurrence_backward(r["h"], r["f"], r["chunk"], r["dy"], r["dx"], r["df"], r["dg"], gate=r["g"], cu_seqlens=cu,
                                            initial_state=r["s0"], grad_initial_state=r["d0"], stream=s)
        A.attnres_layer_norm_backward(r["x"], r["dx"], r["dh"], r["gain"], r["gg"], r["gb"], workspace=r["ws"], stream=s)
        A.attnres_grad_clip([r["gg"], r["gb"], r["dh"]], 0.5, r["norm"], workspace=r["cws"], stream=s)

    names = ("out", "fin", "chunk", "dx", "df", "dg", "d0", "dh", "gg", "gb", "norm")
    sets = [make(1), make(2)]
    want = []
    for r in sets:
        call(r, None)
        torch.cuda.synchronize()
        want.append([r[k].clone() for k in names])
        for k in names:
            r[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        for r, s in zip(sets, streams):
            call(r, s)
    torch.cuda.synchronize()
    for r, w in zip(sets, want):
        for k, v in zip(names, w):
            assert torch.equal(r[k], v), k
