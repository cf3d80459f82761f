/*
 * tlrgemm.h - Tile-Low-Rank GEMM with a dense output on AMD Instinct MI355X (gfx950).
 *
 *   C <- alpha * op(A) * op(B) + beta * C,   C dense, A TLR, B TLR or dense.
 *
 * The operation is the one stated in the introduction of "Tile-Low-Rank GEMM:
 * Designing Storage Around the Contraction" (dense C, one or both operands in
 * TLR format, op in {N, T}).  A TLR matrix is a regular grid of b x b tiles
 * (the last tile row / column is smaller when b does not divide the
 * dimension); diagonal tiles may be stored densely, every other tile (i,j) is
 * a factor pair U_ij V_ij^T of its own rank r_ij ("TLR Matrix
 * Multiplication", section "Introduction: TLR GEMM").
 *
 * Storage (section "Packing for the contraction" of the first page):
 *   outer  U: packed by tile row.  Column-major, leading dimension b.  Tile
 *             (i,j) occupies r_ij consecutive columns starting at column
 *             sum_{i'<i} rho_i' + sum_{j'<j} r_ij'      (rho_i = sum_j r_ij),
 *             of which its first s_i rows are used.
 *   inner  V: packed by tile column.  Column-major, leading dimension b.  Tile
 *             (i,j) occupies r_ij consecutive columns starting at column
 *             sum_{j'<j} kappa_j' + sum_{i'<i} r_i'j    (kappa_j = sum_i r_ij),
 *             of which its first s_j rows are used.
 *   diag   D: q slots of b*b elements; slot i holds tile (i,i) column-major
 *             with leading dimension b (top-left s_i x s_i used).  Only when
 *             the matrix is square and has_diag != 0; r_ii must then be 0.
 * Each tile takes exactly r_ij columns: no padding to a common rank.  Because
 * U is packed by tile row and V by tile column, a row panel of U and a column
 * panel of V are ordinary column-major matrices, which is what lets the
 * library fold tile indices into GEMM dimensions without copies.
 * op(X) = X^T is taken by swapping the roles of the two factor families and
 * the tile coordinates (section "Where fusion stops", Transposes); no data
 * moves.
 *
 * Dense matrices (C, a dense B) are column-major with a leading dimension.
 * All element types are float (TLR_F32), double (TLR_F64), IEEE half (TLR_F16)
 * or bfloat16 (TLR_BF16), the same for every buffer of one call.
 *
 * 16-bit types (the half-precision paths of the first page's evaluation, run
 * on the 16-bit matrix cores with float accumulation).  Every stored rank is
 * a multiple of 8: a tile of logical rank r is stored with its rank rounded up
 * to the next multiple of 8, the extra factor columns zero, which leaves the
 * product unchanged and keeps every factor column offset a multiple of 16
 * bytes (section "Packing for the contraction").  The tile size b, the
 * dimensions of A, B and C and the leading dimensions ldb and ldc are
 * multiples of 8 too, and every buffer is 16-byte aligned; analysis rejects
 * anything else with TLR_ERR_INVALID_ARG (TLR_ERR_RANK for a rank), execution
 * rejects a misaligned buffer.  The products are accumulated in float; each
 * workspace intermediate (the coupling blocks, the right or left products)
 * and C are rounded to the 16-bit type once, when written, and alpha and beta
 * are applied in float.  In half precision those intermediates must stay
 * within its range (|x| <= 65504; beyond it they become infinite); bfloat16
 * has float's range.
 *
 * Ownership: every device buffer (factors, diagonals, dense B, C, workspace,
 * descriptor buffer) belongs to the caller.  The library never allocates
 * device memory; the one piece it holds is the static workspace array of
 * tlr_gemm_execute_noalloc (TLR_STATIC_WORKSPACE_BYTES per GPU, part of the
 * loaded code object).  A plan owns host memory and the HIP events it
 * creates; the plan copies the rank tables at analysis time.
 *
 * Errors: every entry point returns a tlr_status and writes its outputs only
 * on TLR_OK.  tlr_last_error() returns a thread-local description of the most
 * recent failure.  Kernel faults are asynchronous and surface at the caller's
 * next synchronisation, as usual for HIP.
 *
 * Streams are passed as opaque pointers (hipStream_t values, e.g.
 * torch.cuda.Stream().cuda_stream under ROCm); NULL means the default stream.
 */
#ifndef TLRGEMM_H
#define TLRGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TLR_OK = 0,
  TLR_ERR_INVALID_ARG = -1,  /* null pointer, bad size, mismatched shapes or leading dims */
  TLR_ERR_RANK = -2,         /* r_ij < 0, r_ij > min(s_i, s_j), or r_ii != 0 with a dense diagonal */
  TLR_ERR_WORKSPACE = -3,    /* budget below what one output tile needs, or workspace too small */
  TLR_ERR_UNSUPPORTED = -4,  /* combination not provided (e.g. forcing the left order with a dense B) */
  TLR_ERR_HIP = -5,          /* a HIP runtime call failed */
  TLR_ERR_NOT_BOUND = -6     /* execute before tlr_plan_bind */
} tlr_status;

/* TLR_E4M3 and TLR_E5M2 (8-bit floating point, the OCP encodings) are the code
 * formats of the block-scaled operators only; the TLR products refuse them. */
typedef enum {
  TLR_F32 = 0, TLR_F64 = 1, TLR_F16 = 2, TLR_BF16 = 3, TLR_E4M3 = 4, TLR_E5M2 = 5
} tlr_dtype;
typedef enum { TLR_OP_N = 0, TLR_OP_T = 1 } tlr_op;
typedef enum { TLR_ORDER_RIGHT = 0, TLR_ORDER_LEFT = 1 } tlr_order;

/* Flags of tlr_gemm_analyze / tlr_gemm_workspace_bytes. */
#define TLR_PLAN_FORCE_RIGHT 0x1u  /* every rectangle uses U (S Z^T) */
#define TLR_PLAN_FORCE_LEFT  0x2u  /* every rectangle uses (U S) Z^T (TLR x TLR only) */
#define TLR_PLAN_NO_REGIONS  0x4u  /* do not split boundary regions onto their own streams */
#define TLR_PLAN_VALIDATE    0x8u  /* also run the exhaustive descriptor self-check (slow; for tests) */
#define TLR_PLAN_PIPELINE    0x10u /* two arenas on two streams: stages 1-2 of one rectangle run beside
                                      stage 3 of the previous one (needs n_streams >= 2) */
#define TLR_PLAN_PER_K       0x20u /* the per-contraction-tile loop instead ("Many small GEMMs"): for
                                      each k, the coupling V_ik^T W_kj, the right product S Z_kj^T
                                      and the update C_ij += U_ik T of every output tile, one pass
                                      over C per k (TLR x TLR only; a comparator: with operands
                                      padded to one rank it is the batched-GEMM baseline the page
                                      compares against) */

/* Structure of one stored TLR operand (host data; no device pointers). */
typedef struct {
  int64_t rows, cols;      /* stored dimensions (before op) */
  int32_t b;               /* tile size, >= 1; q_r = ceil(rows/b), q_c = ceil(cols/b) */
  int32_t has_diag;        /* 1: diagonal tiles dense (rows == cols required) */
  const int32_t *ranks;    /* q_r*q_c ranks, column-major: rank of tile (i,j) at ranks[i + j*q_r] */
} tlr_shape;

/* Device buffers of one stored TLR operand, laid out as described above. */
typedef struct {
  const void *diag;        /* NULL iff has_diag == 0 */
  const void *outer;       /* U, packed by tile row;  may be NULL when every rank is 0 */
  const void *inner;       /* V, packed by tile column; may be NULL when every rank is 0 */
} tlr_buffers;

typedef struct tlr_plan tlr_plan;

/* Counts describing a plan (tlr_plan_info). */
typedef struct {
  int64_t m, n, k;             /* C is m x n; the contraction has k columns of op(A) */
  double useful_flops;         /* flops of the method for the chosen orders, from rank metadata */
  double executed_flops;       /* sum over kernel tasks of 2*M*N*K (>= useful when some ranks are 0) */
  double flops_right;          /* whole-C useful flops if every tile used the right order */
  double flops_left;           /* ... the left order (-1 for a dense B) */
  double final_flops_right;    /* 2 sum_i m_i rho_i sum_j n_j */
  double final_flops_left;     /* 2 sum_j n_j gamma_j sum_i m_i (-1 for a dense B) */
  double algorithmic_bytes;    /* compressed A + (compressed or dense) B + C written once (add m*n elements
                                  for the read of C when beta != 0) */
  size_t workspace_bytes;      /* device workspace execute needs (<= the analysis budget) */
  size_t descriptor_bytes;     /* device buffer size tlr_plan_bind needs */
  int32_t runs;                /* output rectangles */
  int32_t groups;              /* region groups (each on its own stream when streams allow) */
  int32_t launches;            /* kernel launches per execute */
  int32_t dtype;               /* tlr_dtype */
} tlr_plan_summary;

/* ---- host-only entry points (no HIP calls) --------------------------------- */

/*
 * tlr_gemm_analyze: build the plan of one product shape ("Association order and
 * workspace": rank prefixes, association order per rectangle, rectangles under
 * the workspace budget, grouped descriptors; reusable for every product with
 * the same rank structure).
 *   dt          element type of every buffer.
 *   opA, A      op and structure of A; A == NULL selects a dense A of
 *               dense_rows x dense_cols (stored, column-major, leading dim ldb):
 *               the dense x TLR product, evaluated in the left order with
 *               op(A) W in place of the coupling (at most one operand dense).
 *   opB, B      op and structure of B; B == NULL selects a dense B of
 *               dense_rows x dense_cols (stored, column-major, leading dim ldb).
 *   ldb         leading dimension of the dense operand (ignored when both are
 *               TLR; < 2^21).
 *   ldc         leading dimension of C (>= m).
 *   workspace_budget  bytes of device workspace execute may use; 0 means no limit.
 *   n_streams   streams execute will be given (>= 1); boundary regions of C
 *               (last tile row / column smaller than b) run concurrently when >= 2.
 *               With TLR_PLAN_PIPELINE the rectangles alternate between two
 *               workspace arenas and streams 0 and 1 ("Association order and
 *               workspace": rectangles write disjoint parts of C, so with two
 *               arenas and two streams the first stages of one rectangle can
 *               overlap the final GEMMs of the previous one, at twice the
 *               workspace); the budget then covers both arenas, and with no
 *               budget each arena is sized for a quarter of C.
 *   flags       TLR_PLAN_* bits.
 *   plan_out    receives a new plan (free with tlr_plan_destroy).
 * Every plan is checked before it is returned: each operand and output range a
 * kernel task can touch must lie inside the buffer sizes the layout above
 * implies (factor buffers b * sum(r_ij) elements, diagonal q*b*b, dense
 * operand ldb * cols, C ldc * n, workspace workspace_bytes); with TLR_PLAN_VALIDATE it
 * also checks that writes inside one launch never overlap, that every
 * workspace element a launch reads was written earlier for the same output
 * rectangle, and that each element of C is written exactly once.
 * Errors: TLR_ERR_INVALID_ARG (shapes, tile sizes or leading dims inconsistent),
 * TLR_ERR_RANK, TLR_ERR_WORKSPACE (budget below one output tile's needs),
 * TLR_ERR_UNSUPPORTED.
 */
tlr_status tlr_gemm_analyze(tlr_dtype dt, tlr_op opA, const tlr_shape *A,
                            tlr_op opB, const tlr_shape *B,
                            int64_t dense_rows, int64_t dense_cols, int64_t ldb,
                            int64_t ldc, size_t workspace_budget, int32_t n_streams,
                            uint32_t flags, tlr_plan **plan_out);

/*
 * tlr_gemm_workspace_bytes: the smallest budget whose schedule has at most
 * `runs` rectangles (runs >= 1; runs == 1 gives the budget of one rectangle
 * covering all of C), found by bisection over the scheduler
 * ("Association order and workspace": workspace bytes for a target number of
 * runs).  Arguments as for tlr_gemm_analyze.  Errors as for analyze.
 */
tlr_status tlr_gemm_workspace_bytes(tlr_dtype dt, tlr_op opA, const tlr_shape *A,
                                    tlr_op opB, const tlr_shape *B,
                                    int64_t dense_rows, int64_t dense_cols,
                                    int32_t n_streams, uint32_t flags, int32_t runs,
                                    size_t *bytes_out);

/* tlr_plan_info: fill *out.  Plumbing: the pages define no such call; the
 * counts are the rank arithmetic of "Association order and workspace" (useful
 * flops, final-stage costs F_R and F_L) and the sizes this library needs.
 * Errors: TLR_ERR_INVALID_ARG on NULL. */
tlr_status tlr_plan_info(const tlr_plan *p, tlr_plan_summary *out);

/*
 * tlr_plan_rect: rectangle `idx` (0 <= idx < runs) of the schedule
 * (introspection; the rectangles are those of "Association order and
 * workspace", the call itself is plumbing the pages do not define).
 *   out_i32[0..5] = first tile row, end tile row (exclusive), first tile
 *                   column, end tile column, order (tlr_order), group.
 *   ws_bytes      workspace the rectangle uses inside its group's arena.
 *   useful_flops  useful flops of the rectangle.
 */
tlr_status tlr_plan_rect(const tlr_plan *p, int32_t idx, int32_t *out_i32,
                         size_t *ws_bytes, double *useful_flops);

/*
 * tlr_plan_stage_shapes: (M, N, K) triples of the logical GEMMs of one stage of
 * rectangle `rect` (introspection, for checking the plan against the shapes
 * the GEMM page prints; the call is plumbing the pages do not define), in order:
 *   stage 1  one coupling GEMM per contraction tile k ("One product, three
 *            stages", Stage 1): (sum_{i in I} r_ik, sum_{j in J} r_kj, s_k);
 *   stage 3  the final GEMMs: per tile row i (right order) (m_i, sum_J n_j, rho_i),
 *            per tile column j (left order) (sum_I m_i, n_j, gamma_j).
 * Writes min(count, cap) triples to mnk[3*t..3*t+2]; *count = number available.
 */
tlr_status tlr_plan_stage_shapes(const tlr_plan *p, int32_t rect, int32_t stage,
                                 int64_t *mnk, int32_t cap, int32_t *count);

/*
 * tlr_plan_launch: launch `idx` (0 <= idx < launches) of one execute
 * (introspection; plumbing the pages do not define).
 *   out_i32[0..3] = stage, tasks, workgroups, group.  Stages: 1 coupling,
 *   2 right/left product, 3 final update, 4 the diagonal-term products that
 *   read only the inputs (X = op(D_A) W or X' = V^T op(D_B), and the op(D_A) W
 *   or op(D_B)^T V blocks of the terminal matrices; the "easy terms" of "TLR
 *   Matrix Multiplication"), run on a side stream beside stages 1 and 2.
 *   out_f64[0..1] = useful flops, executed flops of the launch.
 */
tlr_status tlr_plan_launch(const tlr_plan *p, int32_t idx, int32_t *out_i32, double *out_f64);

/* tlr_plan_destroy: free the plan and its events (NULL is accepted).  Plumbing:
 * the pages define no such call. */
tlr_status tlr_plan_destroy(tlr_plan *p);

/* ---- device entry points ------------------------------------------------- */

/*
 * tlr_plan_bind: copy the plan's descriptor tables into `dev_desc`, a caller
 * device buffer of at least descriptor_bytes bytes (256-byte aligned), on
 * `stream`, and create the plan's fork/join events on the current device.
 * The buffer must stay alive and unmodified while the plan is executed.
 * Plumbing the pages do not define: the GEMM page only says that this setup
 * is done once per rank structure and skipped afterwards ("Association order
 * and workspace").
 * Errors: TLR_ERR_INVALID_ARG (NULL, too small, misaligned), TLR_ERR_HIP.
 */
tlr_status tlr_plan_bind(tlr_plan *p, void *dev_desc, size_t bytes, void *stream);

/*
 * tlr_gemm_execute: C <- alpha op(A) op(B) + beta C with the bound plan: the
 * BLAS-style operation of the GEMM page's introduction, with a dense C and one
 * or both operands in TLR format ("Tile-Low-Rank GEMM: Designing Storage
 * Around the Contraction", introduction), evaluated in the three stages of
 * "One product, three stages" (coupling, right or left product, one update of
 * C with the sum over k inside the GEMM) and with the diagonal terms of "TLR
 * Matrix Multiplication", "Regular TLR GEMM".
 *   A, B        device buffers of the analysed TLR operands (NULL for the
 *               dense one).
 *   B_dense     the dense operand (dense A or dense B as analysed), leading
 *               dim ldb; NULL when both operands are TLR.
 *   C           m x n column-major, leading dim ldc (both as analysed).
 *   workspace   device buffer of at least workspace_bytes (256-byte aligned).
 *   streams     n_streams >= 1 streams; streams[0] is the caller's: the call is
 *               ordered after earlier work on streams[0] and later work on
 *               streams[0] is ordered after it.  Other streams are forked from
 *               and joined back to streams[0] with events.
 * beta == 0 never reads C (NaN in C does not propagate); alpha == 0 only scales C.
 * Asynchronous: no host synchronisation.
 * 16-bit types: every buffer (factors, diagonals, dense operand, C, workspace)
 * must be 16-byte aligned.
 * Errors: TLR_ERR_NOT_BOUND, TLR_ERR_INVALID_ARG (NULL buffers, ld mismatch,
 * a 16-bit buffer off a 16-byte boundary; nothing is launched),
 * TLR_ERR_WORKSPACE (workspace too small), TLR_ERR_HIP (launch failure).
 */
tlr_status tlr_gemm_execute(tlr_plan *p, double alpha,
                            const tlr_buffers *A, const tlr_buffers *B,
                            const void *B_dense, int64_t ldb,
                            double beta, void *C, int64_t ldc,
                            void *workspace, size_t workspace_bytes,
                            void *const *streams, int32_t n_streams);

/* Bytes of the static device workspace of tlr_gemm_execute_noalloc (per GPU). */
#define TLR_STATIC_WORKSPACE_BYTES (256u * 1024u * 1024u)

/*
 * tlr_gemm_execute_noalloc: tlr_gemm_execute without a workspace argument,
 * for callers that cannot allocate device memory at the call (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).  The
 * same plan runs the same launches; the workspace is the library's own static
 * device array of TLR_STATIC_WORKSPACE_BYTES, one per GPU, which every GPU the
 * library runs on holds until the process ends.  The call allocates nothing
 * (no hipMalloc, hipFree or allocating library routine); the plan must already
 * be bound (tlr_plan_bind, whose descriptor buffer the caller allocates once).
 * Every call on one GPU shares that GPU's array and leaves its last contents
 * in it (no product reads workspace it has not written first, so nothing
 * needs clearing).  Calls on one GPU must be ordered (one stream, or events
 * between them): calls that overlap race on the shared array.
 *   Arguments as for tlr_gemm_execute.
 * Errors: as tlr_gemm_execute; TLR_ERR_WORKSPACE when the plan needs more than
 * TLR_STATIC_WORKSPACE_BYTES (analyse with a budget at most that size);
 * nothing is launched then.
 */
tlr_status tlr_gemm_execute_noalloc(tlr_plan *p, double alpha,
                                    const tlr_buffers *A, const tlr_buffers *B,
                                    const void *B_dense, int64_t ldb,
                                    double beta, void *C, int64_t ldc,
                                    void *const *streams, int32_t n_streams);

/*
 * Profiling (plumbing the pages do not define; it feeds the measurement).
 * tlr_plan_profile: record a HIP event pair around every launch of the next
 * `max_executes` executes (0 switches recording off).  Creates the events on
 * the current device.  Errors: TLR_ERR_HIP.
 * tlr_plan_profile_read: after the caller has synchronised, sum the recorded
 * kernel time per stage into stage_ms[5]: stage_ms[0..2] = stages 1..3,
 * stage_ms[3] = the whole execute (first launch start to last launch end on
 * streams[0]), stage_ms[4] = stage 4 (the side launches, which overlap stages
 * 1 and 2);
 * launch_ms (may be NULL) receives the per-launch sums, `launches` entries.
 * *executes = executes recorded.  Resets the record.
 */
tlr_status tlr_plan_profile(tlr_plan *p, int32_t max_executes);
tlr_status tlr_plan_profile_read(tlr_plan *p, double *stage_ms, double *launch_ms,
                                 int32_t *executes);

/*
 * tlr_dense_gemm: C <- alpha op(A) op(B) + beta C for dense column-major
 * matrices, on the same MFMA kernel (one K segment per output tile).  It is
 * the same-chip dense reference the TLR product is compared with ("Results":
 * dense-GEMM time scaled by the ratio of executed flops).
 *   op(A) is m x k, op(B) is k x n, C is m x n; lda/ldb/ldc >= rows of the
 *   stored matrices, lda and ldb < 2^21.  beta == 0 never reads C.  No workspace.
 *   TLR_F32 and TLR_F64 only.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED (a 16-bit type), TLR_ERR_HIP.
 */
tlr_status tlr_dense_gemm(tlr_dtype dt, tlr_op opA, tlr_op opB, int64_t m, int64_t n,
                          int64_t k, double alpha, const void *A, int64_t lda,
                          const void *B, int64_t ldb, double beta, void *C, int64_t ldc,
                          void *stream);

/* ---- TLR output: expansion and compression --------------------------------
 *
 * "TLR Matrix Multiplication", "Introduction: TLR GEMM": each of A, B and C
 * may be stored densely or in TLR format, and the TLR-output cases extend
 * the dense-output product.  The pages give no algorithm or accuracy target
 * for them; this library reads them as: the exact result tile, then every
 * off-diagonal tile replaced by its truncated SVD of the smallest rank whose
 * discarded part meets a relative Frobenius tolerance tol,
 *     ||X_ij - U_ij V_ij^T||_F <= tol ||X_ij||_F,
 * diagonal tiles kept dense.  A product C <- alpha op(A) op(B) + beta C with
 * a TLR C is then: tlr_expand of C into a dense m x n scratch (alpha = 1,
 * beta = 0; skipped when beta == 0), tlr_gemm_execute into that scratch with
 * the caller's alpha and beta, and tlr_compress of the scratch into the new
 * C.  Only TLR_F32 and TLR_F64; everything runs on `stream` with no host
 * synchronisation, and the ranks of a compressed result stay on the device
 * until the caller copies them.
 */

/*
 * tlr_expand: C <- alpha X + beta C, X the dense matrix of a stored TLR
 * operand (tile (i,j) = U_ij V_ij^T of rank r_ij, dense diagonal tiles when
 * has_diag), C dense rows x cols column-major with leading dim ldc >= rows.
 *   ranks_dev  DEVICE q_r x q_c int32 ranks, column-major (r_ii = 0 with a
 *              dense diagonal): the layout of X's packed factors (as for
 *              tlr_shape.ranks).
 *   X          device buffers of the operand.
 *   workspace  device, at least 16 * q_r * q_c bytes, 8-byte aligned (the
 *              factor offsets, computed on the device).
 * beta == 0 never reads C.  Errors: TLR_ERR_INVALID_ARG, TLR_ERR_WORKSPACE,
 * TLR_ERR_UNSUPPORTED (16-bit types), TLR_ERR_HIP.
 */
tlr_status tlr_expand(tlr_dtype dt, int64_t rows, int64_t cols, int32_t b, int32_t has_diag,
                      const int32_t *ranks_dev, const tlr_buffers *X, double alpha, double beta,
                      void *C, int64_t ldc, void *workspace, size_t workspace_bytes, void *stream);

/* tlr_compress_workspace_bytes: device workspace tlr_compress needs for a
 * rows x cols matrix, tile size b and ranks up to max_rank.  Host only.
 * Errors as for tlr_compress's argument checks. */
tlr_status tlr_compress_workspace_bytes(tlr_dtype dt, int64_t rows, int64_t cols, int32_t b,
                                        int32_t max_rank, size_t *bytes_out);

/*
 * tlr_compress: the dense rows x cols matrix X (column-major, leading dim
 * ldx) as a TLR operand with tile size b: diagonal tiles dense (has_diag,
 * square X), every other tile (i,j) the truncated SVD of the smallest rank
 * r_ij <= max_rank with ||X_ij - U_ij V_ij^T||_F <= tol ||X_ij||_F.
 * Method: a range sketch X_ij Omega with s = max_rank + 8 samples, its QR,
 * the projection X_ij^T Q and its QR, and a one-sided Jacobi SVD of the
 * s x s core; the energy the sketch misses counts as discarded.  The rank is
 * decided on squared singular values, so tol must lie well above the square
 * root of the unit roundoff (fp64: tol >= 1e-7; fp32: tol >= 1e-3); for an
 * input of numerical rank above s - 8 the sketch may miss energy.
 *   omega      device b x s Gaussian sketch (column-major, leading dim b),
 *              drawn by the caller, s = max_rank + 8 (max_rank <= 56).
 *   ranks_out  device q_r x q_c int32, column-major: the new ranks (0 on a
 *              dense diagonal).
 *   diag       device q_r slots of b*b (when has_diag), as in the storage above.
 *   outer, inner  device factor buffers (leading dim b) of `capacity`
 *              columns each; tile (i,j) is written at the packed offsets of
 *              its new rank (U packed by tile row, V by tile column).  U has
 *              orthogonal columns of norms sigma_k, V orthonormal columns.
 *   info       device int32[6]: [0] columns used (sum of the new ranks),
 *              [1] tiles that did not meet tol within max_rank (their rank is
 *              max_rank), [2] 1 when [0] exceeds capacity (then no factor is
 *              written; ranks and diagonal are), [3] Jacobi pair visits
 *              (2 x 2 Gram blocks formed) and [4] Jacobi rotations summed over
 *              the tiles (the SVD's work, for measurement), [5] sketch basis
 *              columns kept, summed over the tiles (the range finder stops
 *              once the sketch shows the rest of a tile negligible; at most
 *              max_rank + 8 per tile); [0], [3], [4], [5] saturate at
 *              INT32_MAX.
 *   workspace  device, tlr_compress_workspace_bytes, 256-byte aligned.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_WORKSPACE, TLR_ERR_UNSUPPORTED (16-bit
 * types, max_rank > 56), TLR_ERR_HIP.
 */
tlr_status tlr_compress(tlr_dtype dt, int64_t rows, int64_t cols, int32_t b, int32_t has_diag,
                        const void *X, int64_t ldx, double tol, int32_t max_rank, const void *omega,
                        int32_t *ranks_out, void *diag, void *outer, void *inner, int64_t capacity,
                        int32_t *info, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Profiling of the compression (plumbing the pages do not define; it feeds the
 * measurement).  tlr_compress_profile: record a HIP event pair, on the call's
 * stream, around each kernel group of the next `max_calls` tlr_compress calls
 * of the process (0 switches recording off).  Errors: TLR_ERR_INVALID_ARG
 * (negative count).
 * tlr_compress_profile_read: after the caller has synchronised, sum the
 * recorded time per group into group_ms[9]: 0 tile norms, 1 sketch products
 * X_t Omega, 2 QR of the sketches, 3 projections X_t^T Q_t, 4 QR of the
 * projections, 5 Jacobi SVD and ranks, 6 factor products, 7 rank scan,
 * 8 packing; *calls = calls recorded.  Resets the record.  Errors:
 * TLR_ERR_HIP when an event has not completed.
 */
tlr_status tlr_compress_profile(int32_t max_calls);
tlr_status tlr_compress_profile_read(double *group_ms, int32_t *calls);

/* ---- block-scaled 8-bit matrices -------------------------------------------
 *
 * A matrix X of `rows` rows and k columns as 8-bit floating point codes with a
 * float scale for each block: X[i,c] ~ scale(i, c) * code[i,c].  Blocks are 128
 * columns wide (the last one narrower) and either 1 or 128 rows high.
 *   codes   code (i,c) at byte i*ld + c (k x rows column-major, as a stored
 *           operand of a T,N product): ld >= k, ld a multiple of 16, codes
 *           16-byte aligned, and every row readable up to k rounded up to 16
 *           (what stands there after column k is never used).
 *   scales  the scale of row block r and column block c at scales[r + c*lds],
 *           lds >= the number of row blocks (rows, or ceil(rows / 128)).
 */
typedef struct {
  const void *codes;
  const float *scales;
  int64_t ld, lds;
  int32_t block;           /* rows of a block: 1 or 128 */
  int32_t fmt;             /* TLR_E4M3 or TLR_E5M2 */
} tlr_block_matrix;

/*
 * tlr_block_quantize: codes and scales of X, of X^T, or of both from one read.
 *   s(block) = max(float(a / top), 2^-100), a the block's largest magnitude and
 *   top the format's largest number (448, 57344);  code = the number of the
 *   format nearest to float(x / s), ties to even.  A block that holds an
 *   infinity or a NaN gets a NaN scale and NaN codes.
 *   dt      TLR_F32, TLR_F16 or TLR_BF16 (X); X[i,c] at element i*ldx + c,
 *           ldx >= k, any alignment of the element type (16-byte aligned rows
 *           load faster).
 *   codes, ldq, scales, lds      the rows x k result (codes NULL: not wanted);
 *           bytes k .. k rounded up to 16 of each row are written as zero.
 *   codes_t, ldq_t, scales_t, lds_t  the k x rows result of X^T (blocks of X^T),
 *           likewise.
 * rows up to 65535 * 128, k up to 2^31 - 1, less than 2^24 tiles of 128 x 128.
 * No workspace.  Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED (TLR_F64),
 * TLR_ERR_HIP.
 */
tlr_status tlr_block_quantize(tlr_dtype dt, tlr_dtype fmt, int32_t block, int64_t rows, int64_t k,
                              const void *X, int64_t ldx, void *codes, int64_t ldq, float *scales,
                              int64_t lds, void *codes_t, int64_t ldq_t, float *scales_t, int64_t lds_t,
                              void *stream);

/* Flags of tlr_block_gemm. */
#define TLR_BLOCK_FAST 0x1u  /* inner sums on the 8-bit matrix instructions (see below) */

/*
 * tlr_block_gemm: C <- alpha A B^T + beta C for block-scaled A (m rows) and B
 * (n rows) with k columns each:
 *   sum over column blocks q of sA(i,q) sB(j,q) sum over c in q of a[i,c] b[j,c],
 * exact products, inner and outer sums in float, C rounded once.
 *   flags   0: the codes are widened to bfloat16 (exactly) and the inner sums
 *           run on the bfloat16 matrix instructions, which add in float.
 *           TLR_BLOCK_FAST: on the 8-bit matrix instructions, at twice their
 *           rate.  Those align the products of one block with the largest of
 *           them and cut each below 2^-13 of its binary order, so that an inner
 *           sum is off by at most 2^-13 of the block's largest |a b| for every
 *           product in it: 1.4e-5 of the result for normally distributed data
 *           (float sums: 7e-8), 5e-5 to 7e-5 where one column of each block is
 *           ten to a hundred times the others on both sides, and without limit
 *           relative to a result that is left after larger products cancel.
 *           For 16-bit results whose operands allow it; never for float ones.
 * C (m x n) is column-major with leading
 * dimension ldc >= m and of type dt (TLR_F32, TLR_F16, TLR_BF16), any
 * alignment of that type.  A linear layer y = x W^T has A = W, B = x, and C
 * row-major over (token, feature); its input gradient takes the transposed
 * codes of W (blocks of 128 rows), its weight gradient two matrices with
 * blocks of 1 row along the tokens.  Any block height on either side.
 * beta == 0 never reads C; alpha == 0 reads neither A nor B.  NaN scales and
 * codes propagate.  The product of two scales is a float of its own: it has to be
 * finite, and loses bits below 2^-126 (e4m3 blocks on both sides that reach no
 * more than about 5e-17).
 *   workspace  device, 256-byte aligned, its contents need not be cleared; what
 *              the call takes (tlr_block_gemm_plan; none where alpha == 0), or
 *              tlr_block_gemm_workspace_bytes, the larger of both modes.  NULL
 *              is fine where that is 0.
 * m and n up to 2^31 - 512 with less than 2^24 tiles of 128 x 128 in C; ld < 2^22.
 * Errors: TLR_ERR_INVALID_ARG (unknown flags among it), TLR_ERR_UNSUPPORTED (dt TLR_F64),
 * TLR_ERR_WORKSPACE, TLR_ERR_HIP.
 */
tlr_status tlr_block_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, size_t *bytes_out);

/* What tlr_block_gemm launches for these sizes (zeros where it launches no
 * product): workgroups of `threads` threads, each `rows` x `cols` of C, in a grid
 * of grid_x x (grid_y * parts); `halves` 2: two halves of a workgroup's waves take
 * alternate column blocks; `parts` > 1: as many pieces of the contraction, added
 * by a second launch.  Depends on the arguments alone. */
typedef struct {
  int32_t rows, cols, threads, halves, parts, reserved;
  int64_t grid_x, grid_y;
  size_t workspace;        /* bytes */
} tlr_block_gemm_choice;
tlr_status tlr_block_gemm_plan(int64_t m, int64_t n, int64_t k, uint32_t flags, tlr_block_gemm_choice *out);

tlr_status tlr_block_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, double alpha,
                          const tlr_block_matrix *A, const tlr_block_matrix *B, double beta, void *C,
                          int64_t ldc, uint32_t flags, void *workspace, size_t workspace_bytes,
                          void *stream);

/* ---- mixture-of-experts layer for a few tokens ------------------------------ */

/* One layer's weights (device) and sizes.  gate_up holds for expert e the rows
 * e*2*inter .. : inter gate rows, then inter up rows, `hidden` entries each;
 * down the rows e*hidden .. of `inter` entries.  Rows are packed (no gaps). */
typedef struct {
  int32_t hidden, inter;       /* multiples of 16, at most 65536 */
  int32_t experts, topk;       /* experts <= 512, topk <= 16, topk <= experts */
  int32_t dt;                  /* TLR_F16 or TLR_BF16: x, router, y, and weights unless wdt is 8-bit */
  int32_t wdt;                 /* dt, or TLR_E4M3: gate_up and down as codes with 128 x 128 block scales */
  int32_t normalize;           /* 1: the chosen experts' probabilities are divided by their sum */
  int32_t reserved;            /* 0 */
  const void *router;          /* experts x hidden, row by row */
  const void *gate_up, *down;  /* 16-byte aligned */
  const float *gate_up_scales; /* per expert ceil(hidden/128) x ceil(2*inter/128), row blocks contiguous */
  const float *down_scales;    /* per expert ceil(inter/128) x ceil(hidden/128) */
} tlr_moe_layer;

/*
 * tlr_moe: for each of `tokens` rows x of X (1 <= tokens <= 256):
 *   l = router x (64-bit sums, so that the choice does not hang on the order
 *   of a sum), prob = softmax(l), the topk experts of the largest l (ties: the
 *   lower index; NaN above all numbers), in decreasing order;
 *   y = sum over the chosen e of prob_e down_e (silu(gate_e x) * (up_e x)),
 *   sums in float, silu(g) u carried to the down product as a sum of two
 *   numbers of type dt: 16 bits of it for bfloat16, 22 for half precision, where
 *   it must stay below 65520, as the TLR products' intermediates, and is cut at
 *   2^-35.  y rounded once.
 *   X, Y     token t at element t*ldx, t*ldy (>= hidden); X rows 16-byte aligned
 *            (ldx a multiple of 8), Y any alignment.
 *   ids      device int32, tokens x topk: the chosen experts; weights: float,
 *            the same shape: their (normalized) probabilities.
 *   workspace  device, tlr_moe_workspace_bytes, 256-byte aligned; cleared by
 *            tlr_moe_init once before its first use, then left as it is: calls
 *            on one workspace are ordered (one stream, or events between them).
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED, TLR_ERR_WORKSPACE, TLR_ERR_HIP.
 */
tlr_status tlr_moe_workspace_bytes(const tlr_moe_layer *layer, int32_t max_tokens, size_t *bytes_out);
tlr_status tlr_moe_init(const tlr_moe_layer *layer, void *workspace, size_t workspace_bytes, void *stream);
tlr_status tlr_moe(const tlr_moe_layer *layer, int32_t tokens, const void *X, int64_t ldx, void *Y,
                   int64_t ldy, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes,
                   void *stream);

/* ---- 8-bit integers with a scale for each row --------------------------------
 *
 * A matrix X of `rows` rows and k columns as 8-bit integers with one float scale
 * for each row: X[i,c] ~ scale(i) * code[i,c].  A weight has a row for each output
 * channel, a batch of activations one for each token.
 *   codes   int8, code (i,c) at byte i*ld + c: ld >= k, ld a multiple of 16, codes
 *           16-byte aligned, and every row readable up to k rounded up to 16 (what
 *           stands there after column k is never used).
 *   scales  the scale of row i at scales[i].
 */
typedef struct {
  const void *codes;
  const float *scales;
  int64_t ld;
} tlr_row_matrix;

/*
 * tlr_row_quantize: codes and scales of X, or of rows picked from it.
 *   s(i) = max(float(a / 127), 2^-100), a the row's largest magnitude;
 *   code = float(x / s) rounded to an integer, ties to even (-127 .. 127).
 *   A row that holds an infinity or a NaN gets a NaN scale and zero codes.
 *   dt      TLR_F32, TLR_F16 or TLR_BF16 (X); X[i,c] at element i*ldx + c,
 *           ldx >= k, any alignment of the element type.
 *   index   NULL: row r of the result is row r of X, which has as many (x_rows).
 *           Otherwise device int32, `rows` of them: row r is row index[r] of X, of
 *           zeros (scale 2^-100) where index[r] is none of 0 .. x_rows - 1.
 *   codes, ldq, scales   the rows x k result; bytes k .. k rounded up to 16 of each
 *           row are written as zero.
 * k up to 2^30.  No workspace.  Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED
 * (TLR_F64), TLR_ERR_HIP.
 */
tlr_status tlr_row_quantize(tlr_dtype dt, int64_t rows, int64_t k, const void *X, int64_t x_rows, int64_t ldx,
                            const int32_t *index, void *codes, int64_t ldq, float *scales, void *stream);

/* Rows of B in consecutive groups, each with an A of its own: rows
 * offsets[g] .. offsets[g + 1] - 1 take the codes at A->codes + g*code_step (bytes,
 * a multiple of 16) with the scales at A->scales + g*scale_step (floats).  offsets is
 * device memory, count + 1 int32 in ascending order within 0 .. n (others are
 * cut to 0 .. n; groups that end before they begin are empty). */
typedef struct {
  const int32_t *offsets;
  int64_t code_step, scale_step;
  int32_t count;           /* 1 .. 1024 */
  int32_t clear;           /* columns of C of no group: 0 left as they are, 1 set to zero */
} tlr_row_groups;

/*
 * tlr_row_gemm: C = A B^T for row-scaled A (m rows: channels) and B (n rows:
 * tokens) with k columns each:
 *   C[i,j] = (float(sum over c of a[i,c] b[j,c]) * sB(j)) * sA(i), rounded to C's
 *   type once.  The sum is exact (32-bit integers); its product with sB(j) is a
 *   float of its own and has to be finite.
 * C (m x n) is column-major with leading dimension ldc >= m and of type dt
 * (TLR_F32, TLR_F16, TLR_BF16), any alignment of that type: a linear layer y = x W^T
 * has A = W, B = x, and C row-major over (token, feature).
 *   groups     NULL, or B's rows in groups with an A each (A's other fields hold
 *              for all of them).
 *   workspace  device, 16-byte aligned, not cleared: tlr_row_gemm_workspace_bytes
 *              for the same sizes.  NULL is fine where that is 0.
 * k up to 131071 (TLR_ERR_UNSUPPORTED above), m and n up to 2^31 - 512 with less than
 * 2^24 tiles of 128 x 128 in C (a group's last tile counts whole); ld < 2^22.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED, TLR_ERR_WORKSPACE, TLR_ERR_HIP.
 */
tlr_status tlr_row_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t groups, size_t *bytes_out);

/* What tlr_row_gemm launches for these sizes (groups 0: none), as
 * tlr_block_gemm_plan. */
tlr_status tlr_row_gemm_plan(int64_t m, int64_t n, int64_t k, int32_t groups, tlr_block_gemm_choice *out);

tlr_status tlr_row_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A,
                        const tlr_row_matrix *B, const tlr_row_groups *groups, void *C, int64_t ldc,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * tlr_row_linear: the same product with B = X (n rows of k entries of type dt, X[j,c]
 * at element j*ldx + c, any alignment of the type), quantized within the call as
 * tlr_row_quantize does: one launch for a few tokens, two or three for more.  C has X's
 * type.
 *   workspace  device, 256-byte aligned, not cleared: tlr_row_linear_workspace_bytes.
 */
tlr_status tlr_row_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, size_t *bytes_out);
tlr_status tlr_row_linear(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const void *X,
                          int64_t ldx, void *C, int64_t ldc, void *workspace, size_t workspace_bytes, void *stream);

/* ---- tokens sorted by expert ------------------------------------------------- */

/*
 * tlr_expert_sort: a row for each of the tokens * topk assignments ids[t,s], such
 * that each expert's rows are consecutive, in the order of the assignments.
 *   ids      device, tokens x topk, int32 or int64 (id_bytes 4 or 8).  An id that is
 *            none of 0 .. experts - 1 belongs to no expert: its rows come last.
 *   offsets  device, experts + 1 int32: expert e has rows offsets[e] .. offsets[e+1]
 *            - 1; rows from offsets[experts] on belong to none.
 *   place    device, tokens x topk int32: the row of each assignment.
 *   rows     device, tokens * topk int32: the token of each row, -1 for rows of no
 *            expert.
 *   workspace  device, 4-byte aligned, not cleared: tlr_expert_sort_workspace_bytes.
 * experts 1 .. 1024, topk 1 .. 64, at most 2^24 assignments.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_WORKSPACE, TLR_ERR_HIP.
 */
tlr_status tlr_expert_sort_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts, size_t *bytes_out);
tlr_status tlr_expert_sort(int32_t id_bytes, int64_t tokens, int32_t topk, int32_t experts, const void *ids,
                           int32_t *offsets, int32_t *place, int32_t *rows, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * Rows of `hidden` entries to the sorted order and back.  dt is TLR_F32, TLR_F16 or
 * TLR_BF16; leading dimensions are at least hidden, any alignment of the type.
 * place as tlr_expert_sort leaves it (values out of range are skipped), end the
 * device address of the first row of no expert (offsets + experts).
 *   gather        Y[place[t,s]] = X[t]; rows of no expert become zeros.
 *   combine       out[t] = sum over s of weights[t,s] Y[place[t,s]], in float in the
 *                 order of s and rounded once; weights NULL: 1.  Rows of no expert
 *                 are not read and add nothing.  With weights NULL it is the
 *                 gradient of gather.
 *   combine_grad  dY[place[t,s]] = weights[t,s] dout[t] (zeros for rows of no
 *                 expert), dweights[t,s] = sum over c of dout[t,c] Y[place[t,s],c]
 *                 (0 for those).  dY or dweights may be NULL; without dweights Y
 *                 is not read.
 * hidden up to 2^24, tokens and topk as for the sort.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED (TLR_F64), TLR_ERR_HIP.
 */
tlr_status tlr_expert_gather(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *X, int64_t ldx,
                             const int32_t *place, const int32_t *end, void *Y, int64_t ldy, void *stream);
tlr_status tlr_expert_combine(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *Y, int64_t ldy,
                              const int32_t *place, const int32_t *end, const float *weights, void *out, int64_t ldo,
                              void *stream);
tlr_status tlr_expert_combine_grad(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *dout,
                                   int64_t ldd, const void *Y, int64_t ldy, const int32_t *place, const int32_t *end,
                                   const float *weights, void *dY, int64_t lddy, float *dweights, void *stream);

/* ---- gated activation with an 8-bit checkpoint -------------------------------- */

/*
 * tlr_gated: Y = silu(g) u for rows of X that hold `inter` entries of g, then as many
 * of u; silu(g) = g / (1 + exp(-g)), in float, Y rounded once.  A far negative gate
 * counts for what it is where the other factors are large, though exp(g) is no normal
 * float: the products with it are in doubles, here and in the gradient.
 *   codes, ldq, scales, lds   NULL, or where the row is kept for the backward pass:
 *           int8 codes of g at codes + 2*i*ldq and of u at codes + (2*i + 1)*ldq,
 *           one scale for every 128 of them (the last ones fewer) at scales + 2*i*lds
 *           and scales + (2*i + 1)*lds.  Scale and codes as tlr_row_quantize's, a
 *           block of 128 in place of a row; bytes inter .. inter rounded up to 16 of
 *           each are written as zero.  ldq >= inter, a multiple of 16, codes 16-byte
 *           aligned; lds >= ceil(inter / 128).
 * tlr_gated_grad: the gradient at the values g', u' that the codes stand for:
 *   dX = (dY u' s (1 + g' (1 - s)), dY g' s), s = 1 / (1 + exp(-g')), rounded once.
 * dt is TLR_F32, TLR_F16 or TLR_BF16 for X, Y and their gradients, any alignment of
 * it; rows * ceil(inter / 128) < 2^31.
 * Errors: TLR_ERR_INVALID_ARG, TLR_ERR_UNSUPPORTED (TLR_F64), TLR_ERR_HIP.
 */
tlr_status tlr_gated(tlr_dtype dt, int64_t rows, int64_t inter, const void *X, int64_t ldx, void *Y, int64_t ldy,
                     void *codes, int64_t ldq, float *scales, int64_t lds, void *stream);
tlr_status tlr_gated_grad(tlr_dtype dt, int64_t rows, int64_t inter, const void *dY, int64_t lddy, const void *codes,
                          int64_t ldq, const float *scales, int64_t lds, void *dX, int64_t lddx, void *stream);

/* Static description of a status code (plumbing; the pages define no error
 * handling). */
const char *tlr_status_string(tlr_status s);
/* Thread-local detail of the last failure on this thread ("" if none; plumbing). */
const char *tlr_last_error(void);
/* Library version string (plumbing). */
const char *tlr_version(void);

#ifdef __cplusplus
}
#endif
#endif /* TLRGEMM_H */
