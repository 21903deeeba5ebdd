"""The bench line's DRAM bytes are those of the sources as they stand: a change of the kernels' code asks for a new
capture, of the AllGather+GEMM kernel and of both orders of GEMM+ReduceScatter."""
import bench


def test_captured_traffic_is_of_the_current_sources():
    h = bench.src_hash(bench.AG_KERNEL_SOURCES)
    for workload in ("ag_70b", "rs_70b", "rs_70b_ring"):
        assert bench.NCU_TRAFFIC[workload].get(h), (workload, h)
