"""The benchmark's captured traffic belongs to the GEMM sources as they stand
(CPU): helpers of other kernels stay out of the files that its hash covers."""
import bench


def test_the_default_workload_reports_its_captured_traffic():
    captured, note = bench.captured_traffic("bf16_fwd_T2560")
    assert captured == bench.GEMM_PAIR_TRAFFIC["bf16_fwd_T2560"]["bytes"], note
