"""CPU tests of what the kernels around drafted tokens rest on: the order of
their synchronisation, where no run can show it."""
import os
import re

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
