"""The stated bounds of the caller's workspaces hold for every size, and are reached (host code only)."""
import tiled_gemm_epilogues_amd as tge


def test_routing_workspace_bound():
    # 2 KiB per expert and 1 KiB more
    reached = False
    for experts in (1, 2, 16, 17, 64, 129, 256, 257, 512, 1000, 1024):
        for rows in (0, 1, 31, 32, 33, 128, 129, 500, 4095, 16384, 16385, 65536, 10 ** 6, 2 ** 26):
            for k in {1, min(8, experts)}:
                st, h = tge.gemm_route_plan_create(rows, experts, k, experts, "f32", 0)
                assert st == tge.STATUS_SUCCESS
                need = tge.gemm_route_workspace_bytes(h)[1]
                assert need <= 2048 * experts + 1024
                reached |= need == 2048 * experts + 1024
                assert tge.gemm_route_plan_destroy(h) == tge.STATUS_SUCCESS
    assert reached


def test_norm_workspace_bound():
    # 2 MiB per 1024 columns
    reached = False
    for N in (1, 8, 1000, 1024, 1025, 4096, 16384, 32768):
        for rows in (0, 1, 7, 300, 5003, 65536, 10 ** 7):
            st, h = tge.gemm_norm_plan_create(rows, N, N, N, "bf16", 1e-5)
            assert st == tge.STATUS_SUCCESS
            need = tge.gemm_norm_workspace_bytes(h)[1]
            assert need <= 2048 * N
            reached |= need == 2048 * N
            assert tge.gemm_norm_plan_destroy(h) == tge.STATUS_SUCCESS
    assert reached
