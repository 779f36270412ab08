/*
 * sgemm_ortho.h -- orthogonalised weight updates (GB300, sm_103a).  Companion
 * of sgemm_experts.h, whose weight gradients it takes: same status codes,
 * types, streams and error behaviour.  The entries take no device memory: the
 * scratch, which is several times an update's size, is the caller's.
 *   ORTHO-NON-ALLOCATING: sgemm_orthogonalize sgemm_orthogonalize_workspace
 */
#ifndef GB300_SGEMM_ORTHO_H
#define GB300_SGEMM_ORTHO_H

#include <stdint.h>

#include "sgemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Added to the type bf16, of an update: quick products (see the accuracy below). */
enum { SGEMM_ORTHO_QUICK = 256 };

/*
 * sgemm_orthogonalize -- E matrices (M x N) with their singular values brought
 * near 1 by Newton-Schulz products:
 *
 *     X = G / (|G|_F + eps),   then `steps` times
 *     A = X X^T,  X = a X + (b A + c A A) X      (X^T X where M > N),
 *
 * which takes each singular value s to a s + b s^3 + c s^5 and leaves the
 * singular vectors where they are.
 *   type       of G and out; SGEMM_ORTHO_QUICK may be added to SGEMM_TYPE_BF16, and to no other
 *   G, ldg, stride_g       E matrices M x N, stride_g elements apart; E up to 2^27 - 1, M and N up to
 *              262144 (sums over longer rows lose more than what follows)
 *   out, ldo, stride_out   the same, overwritten
 *   steps      1 .. 64
 *   a, b, c    the polynomial.  It may take no singular value that can occur
 *              (from [0, 1] on) above 2 in magnitude after any step, and
 *              b s^2 + c s^4 not above 15: refused otherwise
 *   eps        >= 0, finite.  With eps = 0 a matrix of zeros gives NaN
 *   workspace  DEVICE memory of workspace_bytes, at least what
 *              sgemm_orthogonalize_workspace says, 256-byte aligned, for this call alone until
 *              its work on the stream is done (NULL where it says 0)
 * Accuracy.  Each step's products take X, A and b A + c A A less their
 * diagonals as two f16 values each (22 bits), three products of which stand for
 * one in float32 (A's and X's rounding errors, and the diagonals, are carried
 * along outside of the products), and sum in float32, whatever the type.  The
 * result is rounded to its type once.  Before that, five steps of the usual
 * polynomials ((3.4445, -4.7750, 2.0315) and those that converge to 1) are off by less
 * than 2^-18 of the result's norm up to rows of 65536, if G has something in
 * all directions.  What rounding leaves in directions where it has nothing is raised
 * by up to a in each step, 485 times in all by the former: 1e-5 of the norm for a
 * rank of 30, up to 2e-4 for one or two, as with float32 products.
 * Many steps of a polynomial that does not converge lose more in any arithmetic: up
 * to 16 times what the same steps with float32 products lose (an accumulator's sum
 * is cut to 24 bits up to 32 times).
 *   SGEMM_ORTHO_QUICK: one f16 value each (11 bits), one product of them for one:
 * a third of the time for large matrices.  Before the rounding to bf16 (1.7e-3 of the
 * norm) five steps of the polynomial above are then off by 4e-4 to 8e-4 (up to 5e-3
 * for a rank of one), ten by 1.6e-3, 64 by 7e-3; nothing is promised
 * for polynomials that raise errors: (3, -1, 0) is off by 2e-2 after six steps and by the norm itself after ten.
 * A non-finite element makes its whole matrix NaN or infinite, and no other.
 */
int sgemm_orthogonalize(int type, int E, int M, int N,
                        const void* G, int64_t ldg, int64_t stride_g,
                        int steps, float a, float b, float c, double eps,
                        void* out, int64_t ldo, int64_t stride_out,
                        void* workspace, int64_t workspace_bytes,
                        void* stream);

/*
 * sgemm_orthogonalize_workspace -- the bytes of workspace that a call of these
 * sizes takes (about 8 an element for several steps, 4 for one, and 8, quick 6, an
 * element of the square of the shorter side; 0 for a shorter side of up to 128 and a longer
 * one of up to 2048), or -1 for sizes that it refuses.  It asks no device (some
 * take longer ones without workspace as well).
 */
int64_t sgemm_orthogonalize_workspace(int type, int E, int M, int N, int steps);

#ifdef __cplusplus
}
#endif
#endif
