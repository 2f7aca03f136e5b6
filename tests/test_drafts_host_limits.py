"""CPU tests of what the kernels around drafted tokens rest on: the order of
their synchronisation, where no run can show it, and arguments that a kernel
could not survive."""
import ctypes
import os
import re

from tensor_relational_einsum_gb300 import _abi
from test_cache_host import ARG, BASE, L, batch, cache, rel  # noqa: F401
from test_drafts_host import FAR, rotary_opts

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_relational_einsum_gb300", "csrc", "kernels")


def test_no_store_to_another_cta_before_the_first_cluster_barrier():
    """Another CTA's shared memory is its own only once that CTA has begun, which a cluster barrier says.  In the source's
    order the wait of one stands before the first store, and the barrier's arrival before its wait."""
    text = open(os.path.join(CSRC, "verify.cu")).read()
    body = re.sub(r"//.*", "", text[text.index("verify_kernel("):])
    store = body.index("put_u")
    arrive, wait = (body.find(f"cluster_{x}()") for x in ("arrive", "wait"))
    sync = body.find("cluster_sync()")
    assert 0 <= sync < store or 0 <= arrive < wait < store


def test_no_launch_assumes_a_number_of_sms():
    """Launches take the number of SMs from the device, not one GPU's as a constant."""
    for name in sorted(os.listdir(CSRC)):
        code = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
        assert not re.search(r"\b(148|152|160)\b", code), name


def test_arrays_off_their_boundary_are_refused(L):  # noqa: F811
    """A 4-byte element off its boundary is a fault on the device: no entry point lets one through."""
    far = dict(pages=BASE << 6, starts=BASE << 7, lens=BASE << 8, max_new=8)
    off = [dict(far, **{x: far[x] + o}) for x in ("pages", "starts", "lens") for o in (1, 2, 3)]
    at = [BASE + i * FAR for i in range(12)]
    c = cache(L)[1]
    # rotary
    q, qo = (rel(L, "bf16", (10, 6, 64), at=at[i]) for i in (0, 1))

    def turn(b=None, **kw):
        o, keep = rotary_opts(**kw)
        return L.ea_rotary(ctypes.byref(o), ctypes.byref(batch(**b)) if b else None, q, None, qo, None, None)

    for o in (1, 2):
        assert turn(positions=(BASE << 9) + o) == ARG and turn(far, parents=(BASE << 9) + o) == ARG
    assert all(turn(b) == ARG for b in off if b["pages"] == far["pages"])
    # verification
    target = rel(L, "f32", (10, 100), at=at[0])
    base = dict(tokens=at[2], parents=at[8], accept=at[3], sample=at[4], path=at[5], counts=at[6], picked=at[7])

    def ask(b=far, **kw):
        o = _abi.VerifyOpts(width=10)
        for x, y in {**base, **kw}.items():
            setattr(o, x, y)
        return L.ea_verify_drafts(ctypes.byref(o), ctypes.byref(batch(**b)), target, None, None)

    assert all(ask(**{x: y + o}) == ARG for x, y in base.items() for o in (1, 2, 3))
    assert all(ask(b) == ARG for b in off if b["pages"] == far["pages"])
    # keep
    def keep(b=far, path=BASE << 9, counts=BASE << 10, lens_out=BASE << 11):
        arr = (ctypes.c_void_p * 1)(c.value)
        return L.ea_cache_keep(arr, 1, ctypes.byref(batch(**b)), path, 8, counts, lens_out, None)

    assert keep(path=(BASE << 9) + 2) == ARG and keep(counts=(BASE << 10) + 1) == ARG and keep(lens_out=(BASE << 11) + 3) == ARG
    assert all(keep(b) == ARG for b in off)
    # the cache's other calls
    k, v, o = rel(L, "bf16", (10, 2, 64), at=at[2]), rel(L, "bf16", (10, 2, 64), at=at[3]), rel(L, "bf16", (10, 6, 64), at=at[4])
    need = ctypes.c_size_t()
    for b in off:
        b = ctypes.byref(batch(**b))
        a = _abi.CacheAttnOpts(0.0, 1, None, None, BASE << 9, 1 << 40)
        assert L.ea_cache_append(c, b, k, v, None) == ARG and L.ea_cache_read(c, b, k, v, None) == ARG
        assert L.ea_cache_attention_workspace(c, b, q, ctypes.byref(need)) == ARG
        assert L.ea_cache_attention(c, b, q, ctypes.byref(a), None, o) == ARG
