"""What the source of the 4-bit product has to say for its hand-overs to be sound,
read without a GPU: orderings whose absence no run shows."""
import os
import re

from doubly_stochastic_projection_b200 import build


def _read(name):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())


def test_no_operand_waits_for_word_of_another_cta():
    # a commit orders the tensor work of its thread, not what that thread has
    # waited for: it tells nobody that operands are there, least of all across
    # CTAs.  Barriers are the CTA's own; what others read of its shared memory
    # (the partial sums) lies between cluster barriers
    product, tc5 = _read("mhc_mx4.cu"), _read("tc5.cuh")
    assert "cta_group::2" not in tc5 and "multicast" not in tc5
    assert all(m.startswith("map_rank(tc5::smem_addr(epi") for m in re.findall(r"map_rank\([^)]*\)?", product))
    for bar in re.findall(r"(?:commit|mbar_arrive|mbar_expect_tx)\w*(?:<\w+>)?\(([^;]*);", product):
        assert "map_rank" not in bar, bar


def test_a_wait_that_ran_out_leaves_nothing_in_flight():
    # a role that has no wait left does not learn in its own code that another
    # gave up: what is in flight is waited for behind a barrier of the CTA, by the
    # roles that issue it, whether their own waits ran out or not
    product = _read("mhc_mx4.cu")
    kernel = product[product.index("mx4_product_kernel(const __grid_constant__"):product.index("tmem_free")]
    assert kernel.count("commit(drained)") == 1
    way_out = kernel[kernel.rindex("tc5::fence_before_sync();"):]
    barrier, check, again = (way_out.index(x) for x in ("__syncthreads();", "if (*abort != 0)", "__syncthreads();\n    }"))
    assert barrier < check < again
    drain = way_out[check:again]
    assert "if (!ok)" not in drain and "if (ok)" not in drain
    assert "warp == 0" in drain and "mbar_wait(full(" in drain and "commit(drained)" in drain
    # nor are sums read that may still be in work
    assert re.search(r"if \(ok\) \{\s*tc5::tmem_load", kernel) and kernel.count("tmem_load(") == 1


def test_product_reads_through_the_coherent_path():
    # the product may start while its producer still runs, so nothing that it reads
    # is constant for its lifetime, as the non-coherent loads ask for
    product = _read("mhc_mx4.cu")
    product = product[product.index("struct ProductArgs"):product.index("cudaError_t launch_premap_fwd_mx4")]
    for word in ("ld.global.nc", "__ldg", "load_maps", "load16", "__restrict__"):
        assert word not in product, word
